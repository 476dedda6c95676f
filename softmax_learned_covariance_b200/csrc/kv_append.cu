// kv_append.cu -- new keys and values into a paged cache (e4m3 with block
// exponents, or bf16).
//
// Token i of sequence b goes to position seqlens[b] + i.  e4m3: the block of 16
// tokens a position falls into takes the exponent e' = max(e of its rows that
// are there, e(largest |x| of its new rows)), e(a) the smallest e with
// a <= 448 2^e, and holds round(x 2^-e'); rows that are there are moved from e
// to e' (exact until subnormal).  Elements that are not finite are stored as
// NaN and do not enter e(a).
//
// One warp per (b, kvh, block, K or V): it owns the block's rows and exponent,
// so nothing is shared between warps.  The 16 x d bf16 rows stay in registers
// between the maximum and the conversion, so x is read once: bound by HBM (4 bytes
// read and 2 written per K/V element pair).  B=8, 16 heads, 4096 tokens, d = 128:
// 66 us a call, 61.5 the kernel (0.40 GB, 6.55 TB/s of 6.57).
#include "cache_common.cuh"

namespace plx {
namespace {

constexpr int WARPS = 4;

// smallest e with a <= 448 2^e for the bf16 magnitude a (finite bits), in [KV_EMIN, KV_EMAX]
__device__ __forceinline__ int exponent_of(uint32_t a) {
    if (a == 0) return KV_EMIN;
    const int e = (int)(a >> 7) - 127 - 8 + ((a & 0x7fu) > 0x60u);   // 448 = 1.75 2^8
    return min(max(e, KV_EMIN), KV_EMAX);
}

__device__ __forceinline__ uint32_t absmax2(uint4 w) {
    return __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
}
// infinities and NaN of a packed pair as 0 (for the maximum) or as NaN (to be stored)
__device__ __forceinline__ uint32_t finite_or(uint32_t w, uint32_t other) {
    if ((w & 0x7f80u) == 0x7f80u) w = (w & 0xffff0000u) | other;
    if ((w & 0x7f800000u) == 0x7f800000u) w = (w & 0xffffu) | other << 16;
    return w;
}

__device__ __forceinline__ uint32_t cvt4(uint32_t a, uint32_t b, float f) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(__uint_as_float(a << 16) * f), "f"(__uint_as_float(a & 0xffff0000u) * f), "f"(__uint_as_float(b << 16) * f),
          "f"(__uint_as_float(b & 0xffff0000u) * f));
    return r;
}

template <int D, bool Q8>
__global__ void __launch_bounds__(WARPS * 32) k_kv_append(KvAppendArgs A, unsigned units, unsigned nblocks, int *__restrict__ err) {
    constexpr int CH = D / 8;             // 16-byte chunks of a bf16 row
    constexpr int RPI = 32 / CH;          // rows per warp load
    constexpr int LOADS = KV_BLOCK / RPI;
    const int lane = threadIdx.x % 32;
    const unsigned u = blockIdx.x * WARPS + threadIdx.x / 32;
    if (u >= units) return;
    const bool is_v = u & 1;
    const int blk = (int)((u >> 1) % nblocks);
    const unsigned bk = (u >> 1) / nblocks;
    const int b = (int)(bk / (unsigned)A.pg.Hkv), kvh = (int)(bk % (unsigned)A.pg.Hkv);
    const int ps = 1 << A.pg.pshift, cap = A.pg.max_pages << A.pg.pshift;
    const int start = min(max(A.seqlens[b], 0), cap);
    int n = A.counts ? min(max(A.counts[b], 0), A.T) : A.T;
    const bool over = n > cap - start;
    if (over) n = cap - start;
    if (kvh == 0 && blk == 0 && !is_v && lane == 0) {
        if (over) atomicExch(err, PARALLAX_ERR_DEVICE_INDEX);
        if (A.new_seqlens) A.new_seqlens[b] = start + n;
    }
    if (n == 0 || blk > (start + n - 1) / KV_BLOCK - start / KV_BLOCK) return;   // no new row
    const int p0 = (start / KV_BLOCK + blk) * KV_BLOCK;      // the block's first position
    const int lo = max(start - p0, 0), hi = min(start + n - p0, KV_BLOCK);   // its new rows
    // the accumulator is the sequence's: its new entries are cleared whatever the page
    if (A.wacc != nullptr && is_v && lane >= lo && lane < hi) A.wacc[(size_t)bk * cap + p0 + lane] = 0.f;
    const int id = A.pg.table[(size_t)b * A.pg.max_pages + (p0 >> A.pg.pshift)];
    if ((unsigned)id >= (unsigned)A.pg.num_pages) {
        if (lane == 0) atomicExch(err, PARALLAX_ERR_DEVICE_INDEX);
        return;
    }
    const size_t slab = (size_t)id * A.pg.Hkv + kvh;
    const int row0 = p0 & (ps - 1);

    const __nv_bfloat16 *x = is_v ? (const __nv_bfloat16 *)A.v : (const __nv_bfloat16 *)A.k;
    const long long sb = is_v ? A.v_stride[0] : A.k_stride[0], sh = is_v ? A.v_stride[1] : A.k_stride[1],
                    st = is_v ? A.v_stride[2] : A.k_stride[2];
    const int ch = lane % CH, rr = lane / CH;
    const __nv_bfloat16 *src = x + b * sb + kvh * sh + ch * 8;
    uint4 w[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = i * RPI + rr;
        w[i] = row >= lo && row < hi ? ldg_nc16(src + (long long)(p0 + row - start) * st) : make_uint4(0u, 0u, 0u, 0u);
    }
    uint8_t *pages = static_cast<uint8_t *>(is_v ? A.vpages : A.kpages);
    if constexpr (!Q8) {
        uint8_t *dst = pages + (slab * ps + row0) * (D * 2) + ch * 16;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int row = i * RPI + rr;
            if (row >= lo && row < hi) *reinterpret_cast<uint4 *>(dst + row * (D * 2)) = w[i];
        }
        return;
    }
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) big = __vmaxu2(big, absmax2(w[i]));
    big = max(big & 0xffffu, big >> 16);
    if (big >= 0x7f80u) {
        big = 0;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const uint4 f = make_uint4(finite_or(w[i].x, 0u), finite_or(w[i].y, 0u), finite_or(w[i].z, 0u), finite_or(w[i].w, 0u));
            const uint32_t m = absmax2(f);
            big = max(big, max(m & 0xffffu, m >> 16));
            w[i] = make_uint4(finite_or(w[i].x, 0x7fc0u), finite_or(w[i].y, 0x7fc0u), finite_or(w[i].z, 0x7fc0u),
                              finite_or(w[i].w, 0x7fc0u));
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off /= 2) big = max(big, __shfl_xor_sync(0xffffffffu, big, off));
    int e = exponent_of(big);
    signed char *ep = (is_v ? A.vexp : A.kexp) + slab * (ps / KV_BLOCK) + row0 / KV_BLOCK;
    uint8_t *dst = pages + (slab * ps + row0) * D;
    if (lo > 0) {
        const int was = *ep;
        e = max(e, was);
        if (e > was) {
            for (int c = lane; c < lo * (D / 16); c += 32) {
                uint4 *p = reinterpret_cast<uint4 *>(dst) + c;
                *p = e4m3_shift_down(*p, e - was);
            }
        }
    }
    __syncwarp();      // every lane has read the old exponent
    if (lane == 0) *ep = (signed char)e;
    const float f = exp2_whole(-e);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = i * RPI + rr;
        if (row >= lo && row < hi)
            *reinterpret_cast<uint2 *>(dst + row * D + ch * 8) = make_uint2(cvt4(w[i].x, w[i].y, f), cvt4(w[i].z, w[i].w, f));
    }
}

template <int D, bool Q8> cudaError_t launch_t(const KvAppendArgs &A, int *err, cudaStream_t s) {
    const unsigned nblocks = (unsigned)(A.T + KV_BLOCK - 1 + KV_BLOCK - 1) / KV_BLOCK;    // blocks T tokens can touch
    const unsigned units = (unsigned)A.B * A.pg.Hkv * nblocks * 2;                        // below 2^31 (checked at entry)
    k_kv_append<D, Q8><<<(units + WARPS - 1) / WARPS, WARPS * 32, 0, s>>>(A, units, nblocks, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &A, const DeviceCtl &ctl, cudaStream_t s) {
    if (A.d == 64) return A.kexp ? launch_t<64, true>(A, ctl.err, s) : launch_t<64, false>(A, ctl.err, s);
    return A.kexp ? launch_t<128, true>(A, ctl.err, s) : launch_t<128, false>(A, ctl.err, s);
}

}  // namespace plx
