// decode_cache.cu -- paged decode over an e4m3 or bf16 cache, with or without a
// probe, that can also add up the attention each cached token receives.
//
// Per query head the operator of the paged decode (zubnet.ai news item on
// Parallax, paragraph 2): z_t = q.k_t / sqrt(d), a_t = rho.k_t, s = softmax(z),
// y = o - (m - o abar); without a probe y = o.  With an accumulator,
// wacc[b, kvh, t] += sum over the KV head's query heads of s_t.
//
// Layout.  Tokens are the rows (M = 16) of both tensor-core products and the
// vectors that share a KV head their 8 columns:
//   [z a] (16 tokens x 8)  = K (16 x d)  x  [q_0 rho_0 .. q_3 rho_3] (d x 8)
//   [O M]^T (d x 8)       += V^T (d x 16 tokens) x [p_0 pa_0 .. p_3 pa_3] (16 x 8)
// so four heads with their probes (or eight without) fill one n-tile: with
// tokens as columns the 16-row operand would be half empty up to four heads
// (half the accumulators and MMAs here).  The score product leaves z and a of
// a (token, head) in one thread, and one movmatrix per 8 tokens turns the
// weights into the second product's operand.
//
// Each warp streams its own 16-token tiles through a ring in shared memory that
// bulk copies (TMA) fill: K and V in four pieces of four tokens each, 32 bytes
// apart from multiples of 128, which makes the threads' 16-byte reads free of
// bank conflicts.  The order of the contracted index is free as long as both
// operands agree, so a thread reads whole 16-byte chunks and uses them as its
// part of the fragments (K: chunks of its own two tokens; V: the same chunk of
// its four tokens): no ldmatrix and no barrier beyond the warp's own mbarriers.
// The loads bound the kernel and how they are issued decides their rate (B=64,
// 16 heads of their own, 4096 tokens, d = 128, 1.07 GB; loads alone): 16-byte
// cp.async in fragment order 205 us, in row order 196 us, bulk copies 168 us.
//
// Numerics.  e4m3 codes are exact in fp16; q and rho are brought to fp16 by a
// power of two per vector (exact down to 2^-22 of the vector's largest
// element); the block exponents multiply z and a in fp32, and V's enters its
// weight relative to the warp's largest so far.  The weights p and p a are
// carried as two 16-bit parts (fp16 hi + lo, or bf16 hi + lo for a bf16 cache,
// whose V then needs no conversion), 2^-17 or better, so their rounding stays
// far below the cache's own; l and abar sum the fp32 weights.
#include <math.h>

#include <type_traits>

#include "cache_common.cuh"
#include "sm100.cuh"

namespace plx {
namespace {

constexpr int WARPS = 4;
#ifndef Q8_STAGES
#define Q8_STAGES 3
#endif
#ifndef BF_STAGES
#define BF_STAGES 3
#endif
#ifndef MINB
#define MINB 4
#endif
#ifndef UPS
#define UPS 16
#endif
constexpr float MNONE = -1e30f;     // reference of a row that has seen no score
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
// A row's reference moves when a score exceeds it by 2^HEADROOM: p <= 2^4, and
// p a is carried as p (a / 2^4), so |a| up to fp16's range stays finite.
constexpr float HEADROOM = 4.f;
constexpr float ASCALE = 16.f;

__device__ __forceinline__ float fex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// `bytes` (a multiple of 16) from global to shared memory; completion is counted on `bar`
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <bool Q8>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (Q8)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 matrix of 16-bit elements, one row per 4 threads -> its transpose
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// (x, y) as two packed 16-bit pairs: hi = rounded, lo = what the rounding left
template <bool Q8> __device__ __forceinline__ void split_pair(float x, float y, uint32_t &hi, uint32_t &lo) {
    if constexpr (Q8) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const float2 f = __bfloat1622float2(h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}

template <typename Tout> __device__ __forceinline__ void store_y(Tout *p, float v);
template <> __device__ __forceinline__ void store_y<float>(float *p, float v) { *p = v; }
template <> __device__ __forceinline__ void store_y<__nv_bfloat16>(__nv_bfloat16 *p, float v) {
    *p = __float2bfloat16_rn(v);
}

constexpr int BAD = 1 << 16;     // a tile's page id is out of range

// row in its piece of the x-th of a thread's four value tokens: columns 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9
__device__ __forceinline__ constexpr int x_row(int x) { return (x & 1) + 2 * (x >> 1); }

// Shapes of one instantiation.  NT n-tiles of 8 vectors: 4 NT heads with a
// probe, 8 NT without.
template <int D, bool Q8, bool RHO, int NT> struct Shape {
    static constexpr int HEADS = (RHO ? 4 : 8) * NT;     // heads of a unit
    static constexpr int HPT = RHO ? NT : 2 * NT;        // of which a thread holds the state of HPT
    static constexpr int EL = Q8 ? 1 : 2;                // bytes of a cache element
    static constexpr int ROW = D * EL;                   // bytes of a row
    static constexpr int KC = ROW / 64;                  // 16-byte chunks of a K row per thread
    static constexpr int KSTEPS = D / 16;                // MMAs of the score product
    static constexpr int VB = ROW / 8;                   // bytes of a V row per thread
    static constexpr int JS = D / 16;                    // MMAs of the value product
    // state of a warp in the merge: per head m, l, abar, then O[D] (and M[D])
    static constexpr int MSTRIDE = (RHO ? 2 : 1) * D + 4;
    static constexpr int MERGE_BYTES = WARPS * HEADS * MSTRIDE * 4;
    // K or V of 16 tokens: four pieces of four rows, 32 bytes off a multiple of 128
    static constexpr int PIECE = 4 * ROW + 32;
    static constexpr int TILE_BYTES = 2 * 4 * PIECE;
    // Token of a thread's score rows r = 2 m + o and r + 8: row o (and o + 2) of piece m,
    // or, for the odd rows of 128-byte and wider rows, of the piece 64 bytes further in
    // the banks; so the 8 threads of a shared-memory phase read 8 different chunks.
    static constexpr int ODD_PIECE = ROW == 64 ? 0 : 2;
    static constexpr int STAGES = Q8 ? Q8_STAGES : BF_STAGES;            // tiles in flight per warp: STAGES - 1
    static constexpr int RING_BYTES = WARPS * STAGES * TILE_BYTES;
    static constexpr int SMEM = RING_BYTES > MERGE_BYTES ? RING_BYTES : MERGE_BYTES;
};

// Partials of a split unit: O[D] (and M[D]) per (b, h, split); its m, l, abar in `hdr`.
template <int D, bool RHO> constexpr int part_stride() { return (RHO ? 2 : 1) * D; }

template <int D, bool Q8, bool RHO, int NT, typename Tout>
__global__ void __launch_bounds__(WARPS * 32, (NT == 1 ? MINB : 2)) k_decode_cache(
    const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ rho, const uint8_t *__restrict__ kp,
    const uint8_t *__restrict__ vp, const signed char *__restrict__ kexp, const signed char *__restrict__ vexp,
    const int *__restrict__ seqlens, Tout *__restrict__ y, float *__restrict__ lse, int Hq, int chunk, int nsplit,
    long units_per_split, int htiles, PagedKV pg, float *__restrict__ parts, float4 *__restrict__ hdr,
    float *__restrict__ zs, DeviceCtl ctl) {
    using S = Shape<D, Q8, RHO, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    float *merge = reinterpret_cast<float *>(smem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r = lane / 4, t4 = lane % 4;
    const float scale_log2 = LOG2E / sqrtf((float)D);
    const int ps = 1 << pg.pshift, pmask = ps - 1;
    const long units = units_per_split * nsplit;
    __shared__ uint64_t full[WARPS][S::STAGES];
    __shared__ int abort_flag;
    if (threadIdx.x == 0) abort_flag = 0;
    if (lane == 0)
        for (int i = 0; i < S::STAGES; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
    fence_mbar_init();
    __syncthreads();
    const WaitCtl wait{ctl.err, &abort_flag, ctl.wait_ns};
    int stage = 0;               // stage of this warp's next tile
    uint32_t phases = 0;         // parity each stage's barrier completes next

    for (long u = blockIdx.x; u < units; u += gridDim.x) {
        const long ut = u % units_per_split;    // chunk-major
        const int split = (int)(u / units_per_split);
        const int b = (int)(ut / ((long)pg.Hkv * htiles));
        const int rem = (int)(ut % ((long)pg.Hkv * htiles));
        const int kvh = rem / htiles, ht = rem % htiles;
        const int g0 = ht * S::HEADS;
        const int nh = min(S::HEADS, pg.group - g0);
        const long h0 = (long)b * Hq + (long)kvh * pg.group + g0;
        const int Tcap = pg.max_pages << pg.pshift;
        const int L = min(max(seqlens[b], 0), Tcap);
        const int t0 = split * chunk;
        if (t0 >= L && nsplit > 1) continue;
        const int t1 = min(L, t0 + chunk);
        const int ntiles = (t1 - t0 + 15) / 16;

        // ---- the vectors: column n = r of n-tile nt; 4 elements per MMA step ----
        uint32_t qf[NT][S::KSTEPS][2];
        float zfac[S::HPT], afac[S::HPT];    // of the heads whose state this thread holds
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int head = RHO ? nt * 4 + r / 2 : nt * 8 + r;
            const bool live = head < nh;
            const __nv_bfloat16 *src = (RHO && (r & 1) ? rho : q) + (h0 + (live ? head : 0)) * D;
            uint2 w[S::KSTEPS];
            uint32_t big = 0;
#pragma unroll
            for (int s = 0; s < S::KSTEPS; ++s) {
                const int d0 = Q8 ? 64 * (s / 4) + 16 * t4 + 4 * (s % 4) : 32 * (s / 2) + 8 * t4 + 4 * (s % 2);
                w[s] = live ? *reinterpret_cast<const uint2 *>(src + d0) : make_uint2(0u, 0u);
                big = max(big, max(max(w[s].x & 0x7fffu, w[s].x >> 16 & 0x7fffu), max(w[s].y & 0x7fffu, w[s].y >> 16 & 0x7fffu)));
            }
            float inv = 1.f;
            if constexpr (Q8) {
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                // bring the largest element to [2^7, 2^8)
                const int up = min(max(134 - (int)(big >> 7), -110), 110);
                const float f = exp2_whole(up);
                inv = exp2_whole(-up);
#pragma unroll
                for (int s = 0; s < S::KSTEPS; ++s) {
                    const __half2 a = __floats2half2_rn(__uint_as_float(w[s].x << 16) * f,
                                                        __uint_as_float(w[s].x & 0xffff0000u) * f);
                    const __half2 c = __floats2half2_rn(__uint_as_float(w[s].y << 16) * f,
                                                        __uint_as_float(w[s].y & 0xffff0000u) * f);
                    qf[nt][s][0] = *reinterpret_cast<const uint32_t *>(&a);
                    qf[nt][s][1] = *reinterpret_cast<const uint32_t *>(&c);
                }
            } else {
#pragma unroll
                for (int s = 0; s < S::KSTEPS; ++s) {
                    qf[nt][s][0] = w[s].x;
                    qf[nt][s][1] = w[s].y;
                }
            }
            // columns 2 t4 and 2 t4 + 1 of the score product: (z, a) of one head, or z of two
            const float f0 = __shfl_sync(0xffffffffu, inv, 8 * t4), f1 = __shfl_sync(0xffffffffu, inv, 8 * t4 + 4);
            if constexpr (RHO) {
                zfac[nt] = f0 * scale_log2;
                afac[nt] = f1;
            } else {
                zfac[2 * nt] = f0 * scale_log2;
                zfac[2 * nt + 1] = f1 * scale_log2;
            }
        }

        float oacc[NT][S::JS][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < S::JS; ++j) oacc[nt][j][0] = oacc[nt][j][1] = oacc[nt][j][2] = oacc[nt][j][3] = 0.f;
        float mref[S::HPT], lsum[S::HPT], asum[S::HPT];
#pragma unroll
        for (int i = 0; i < S::HPT; ++i) {
            mref[i] = MNONE;
            lsum[i] = asum[i] = 0.f;
        }
        int evref = -1000;        // exponent O and M are held at (e4m3)

        // This warp's tiles are warp + WARPS j.  Lane l holds the page of tile 32 n + l
        // (a tile's rows share one page: it starts on a multiple of 16 and pages hold at
        // least 16) and its two exponents, loaded 32 tiles at a time.
        const int mine = ntiles > warp ? (ntiles - warp + WARPS - 1) / WARPS : 0;
        auto page_of = [&](int j) -> int {
            return j < mine ? pg.table[(size_t)b * pg.max_pages + ((t0 + (warp + WARPS * j) * 16) >> pg.pshift)] : 0;
        };
        // exponents of K (low byte) and V (next byte), and BAD for a page id out of range
        auto info_of = [&](int j, int id) -> int {
            if (j >= mine) return 0;
            if ((unsigned)id >= (unsigned)pg.num_pages) {
                atomicExch(ctl.err, PARALLAX_ERR_DEVICE_INDEX);
                return BAD;
            }
            if constexpr (!Q8) return 0;
            const size_t at = ((size_t)id * pg.Hkv + kvh) * (ps / KV_BLOCK) +
                              ((t0 + (warp + WARPS * j) * 16) & pmask) / KV_BLOCK;
            return (kexp[at] & 0xff) | (vexp[at] & 0xff) << 8;
        };
        int ids = page_of(lane), ids_next = 0, info = info_of(lane, ids), info_next = 0;

        uint8_t *ring = smem + warp * S::STAGES * S::TILE_BYTES;
        // copies tile j from page `id` into stage st, lane l < 8 one piece of K (l < 4) or V;
        // rows past t1, and all rows of a bad page, are left out
        auto issue = [&](int j, int st, int id) {
            const int t = t0 + (warp + WARPS * j) * 16;
            const bool ok = (unsigned)id < (unsigned)pg.num_pages;
            const int rows = ok ? min(16, t1 - t) : 0;
            const uint32_t bar = smem_u32(&full[warp][st]);
            if (lane == 0) mbar_arrive_expect_tx(bar, 2 * rows * S::ROW);
            __syncwarp();
            const int piece = lane & 3, n = min(rows - 4 * piece, 4);
            const bool skip = (ctl.debug_flags & DEBUG_DECODE_SKIP_FIRST_TILE) != 0 && j == 0;
            if (lane < 8 && n > 0 && !skip) {
                const size_t row = (((size_t)id * pg.Hkv + kvh) << pg.pshift) + (t & pmask) + 4 * piece;
                bulk_load(smem_u32(ring + st * S::TILE_BYTES + lane * S::PIECE), (lane < 4 ? kp : vp) + row * S::ROW,
                          n * S::ROW, bar);
            }
        };
#pragma unroll
        for (int j = 0; j < S::STAGES - 1; ++j) {
            const int id = __shfl_sync(0xffffffffu, ids, j);
            if (j < mine) issue(j, (stage + j) % S::STAGES, id);
        }
        // where this thread's tokens and chunks lie in a tile
        const int tok0 = 4 * ((r / 2 + (r & 1) * S::ODD_PIECE) & 3) + (r & 1), tok1 = tok0 + 2;
        const uint32_t koff = (tok0 / 4) * S::PIECE + (tok0 & 3) * S::ROW + 16 * t4;
        const int vpiece[2] = {t4, (t4 + S::ODD_PIECE) & 3};
        const uint32_t voff = (S::VB < 16 ? S::VB : 16) * r;
        for (int j = 0; j < mine; ++j) {
            // ---- pages and exponents of the 32 tiles after these, in good time ----
            if ((j & 31) == 0)
                ids_next = page_of(j + 32 + lane);
            else if ((j & 31) == 16)
                info_next = info_of(j + 16 + lane, ids_next);
            const int jn = j + S::STAGES - 1;
            const int id = __shfl_sync(0xffffffffu, (j & 31) + S::STAGES - 1 < 32 ? ids : ids_next, jn & 31);
            // every lane has read the tile before this one: its stage takes tile jn
            if (jn < mine) issue(jn, stage == 0 ? S::STAGES - 1 : stage - 1, id);
            const int now = __shfl_sync(0xffffffffu, info, j & 31);
            const int ke = (int)(signed char)now, ve = (int)(signed char)(now >> 8);
            if ((j & 31) == 31) {
                ids = ids_next;
                info = info_next;
            }
            const bool landed = mbar_wait(smem_u32(&full[warp][stage]), (phases >> stage) & 1u, wait);
            if (!__all_sync(0xffffffffu, landed)) {
                // give up: let this warp's copies land (bounded) before the CTA's memory goes
                for (int i = j; i < min(jn + 1, mine); ++i) {
                    const int st = (stage + i - j) % S::STAGES;
                    mbar_wait_drain(smem_u32(&full[warp][st]), (phases >> st) & 1u, 2000000ull);
                }
                break;
            }
            phases ^= 1u << stage;
            const uint8_t *dk = ring + stage * S::TILE_BYTES, *dv = dk + 4 * S::PIECE;
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
            const int tile = t0 + (warp + WARPS * j) * 16;
            const int nvalid = t1 - tile;                   // tokens of the tile
            const int nread = now & BAD ? 0 : nvalid;       // rows of it that were copied

            // ---- scores ----
            float sc[NT][4], sc2[NT][4];          // two chains of products
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[nt][e] = sc2[nt][e] = 0.f;
#pragma unroll
            for (int c = 0; c < S::KC; ++c) {
                uint4 k0 = *reinterpret_cast<const uint4 *>(dk + koff + 64 * c);
                uint4 k1 = *reinterpret_cast<const uint4 *>(dk + koff + 2 * S::ROW + 64 * c);
                if (nread < 16) {                           // what was not copied is not looked at
                    if (tok0 >= nread) k0 = make_uint4(0u, 0u, 0u, 0u);
                    if (tok1 >= nread) k1 = make_uint4(0u, 0u, 0u, 0u);
                }
                const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int i = 0; i < (Q8 ? 4 : 2); ++i) {
                    const int st = c * (Q8 ? 4 : 2) + i;
                    uint32_t a0, a1, a2, a3;
                    if constexpr (Q8) {
                        e4m3x4_to_f16x2(w0[i], a0, a2);
                        e4m3x4_to_f16x2(w1[i], a1, a3);
                    } else {
                        a0 = w0[2 * i];
                        a2 = w0[2 * i + 1];
                        a1 = w1[2 * i];
                        a3 = w1[2 * i + 1];
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816<Q8>(st % 2 ? sc2[nt] : sc[nt], a0, a1, a2, a3, qf[nt][st][0], qf[nt][st][1]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[nt][e] += sc2[nt][e];

            // ---- weights ----
            float f[S::HPT], dz[S::HPT][2];       // score = sc * f; dz: against the reference
            bool up = Q8 && ve > evref;
            const float kscale = Q8 ? exp2_whole(ke) : 1.f;
#pragma unroll
            for (int h = 0; h < S::HPT; ++h) {
                const int nt = RHO ? h : h / 2, e = RHO ? 0 : h % 2;
                f[h] = Q8 ? fminf(zfac[h] * kscale, 3e38f) : zfac[h];     // finite: a score of 0 stays 0
                dz[h][0] = fmaf(sc[nt][e], f[h], -mref[h]);
                dz[h][1] = fmaf(sc[nt][2 + e], f[h], -mref[h]);
                if (nvalid < 16) {
                    if (tok0 >= nvalid) dz[h][0] = -INFINITY;
                    if (tok1 >= nvalid) dz[h][1] = -INFINITY;
                }
                up |= fmaxf(dz[h][0], dz[h][1]) > HEADROOM;
            }
            if (zs != nullptr) {
                float *dst = zs + ((((size_t)b * pg.Hkv + kvh) * htiles + ht) * (size_t)Tcap + tile) * S::HEADS;
#pragma unroll
                for (int h = 0; h < S::HPT; ++h) {
                    const int nt = RHO ? h : h / 2, e = RHO ? 0 : h % 2;
                    const int head = RHO ? 4 * h + t4 : 8 * (h / 2) + 2 * t4 + h % 2;
                    if (tok0 < nvalid) dst[tok0 * S::HEADS + head] = sc[nt][e] * f[h];
                    if (tok1 < nvalid) dst[tok1 * S::HEADS + head] = sc[nt][2 + e] * f[h];
                }
            }
            if (__any_sync(0xffffffffu, up)) {
                const float vshift = Q8 ? fex2((float)min(evref - ve, 0)) : 1.f;
                evref = max(evref, ve);
#pragma unroll
                for (int h = 0; h < S::HPT; ++h) {
                    const int nt = RHO ? h : h / 2, e = RHO ? 0 : h % 2;
                    float z0 = sc[nt][e] * f[h], z1 = sc[nt][2 + e] * f[h];
                    if (tok0 >= nvalid) z0 = -INFINITY;
                    if (tok1 >= nvalid) z1 = -INFINITY;
                    float mx = fmaxf(z0, z1);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float mnew = fmaxf(mref[h], mx);
                    const float alpha = fex2(mref[h] - mnew);
                    mref[h] = mnew;
                    dz[h][0] = z0 - mnew;
                    dz[h][1] = z1 - mnew;
                    lsum[h] *= alpha;
                    asum[h] *= alpha;
                    const float beta = alpha * vshift;
#pragma unroll
                    for (int i = 0; i < S::JS; ++i) {
                        if constexpr (RHO) {
                            oacc[nt][i][0] *= beta;
                            oacc[nt][i][1] *= beta;
                            oacc[nt][i][2] *= beta;
                            oacc[nt][i][3] *= beta;
                        } else {
                            oacc[nt][i][e] *= beta;
                            oacc[nt][i][2 + e] *= beta;
                        }
                    }
                }
            }
            const float vfac = Q8 ? fex2((float)(ve - evref)) : 1.f;
            uint32_t bh[NT][2], bl[NT][2];    // weights as the value product's operand: hi, lo parts
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w0, w1;
                    if constexpr (RHO) {
                        // masked tokens have p = 0 and, their K rows being zero, a = 0
                        const float p = fex2(dz[nt][x]);
                        const float a = sc[nt][2 * x + 1] * (Q8 ? fminf(afac[nt] * kscale, 3e38f) : afac[nt]);
                        lsum[nt] += p;
                        asum[nt] = fmaf(p, a, asum[nt]);
                        w0 = p * vfac;
                        w1 = w0 * (a * (1.f / ASCALE));
                    } else {
                        w0 = fex2(dz[2 * nt][x]);
                        w1 = fex2(dz[2 * nt + 1][x]);
                        lsum[2 * nt] += w0;
                        lsum[2 * nt + 1] += w1;
                        w0 *= vfac;
                        w1 *= vfac;
                    }
                    uint32_t hi, lo;
                    split_pair<Q8>(w0, w1, hi, lo);
                    bh[nt][x] = movmatrix(hi);
                    bl[nt][x] = movmatrix(lo);
                }
            // ---- O += P V, M += (P o A) V ----
#pragma unroll
            for (int c = 0; c < (S::VB + 15) / 16; ++c) {
                uint32_t v[4][4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {       // tokens of the weights' columns 2 t4, 2 t4 + 1, + 8, + 9
                    const uint8_t *src = dv + vpiece[x & 1] * S::PIECE + x_row(x) * S::ROW + voff + 128 * c;
                    if constexpr (S::VB < 16) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(src);
                        v[x][0] = w.x;
                        v[x][1] = w.y;
                    } else {
                        const uint4 w = *reinterpret_cast<const uint4 *>(src);
                        v[x][0] = w.x;
                        v[x][1] = w.y;
                        v[x][2] = w.z;
                        v[x][3] = w.w;
                    }
                    if (nread < 16 && 4 * vpiece[x & 1] + x_row(x) >= nread) v[x][0] = v[x][1] = v[x][2] = v[x][3] = 0u;
                }
                constexpr int PER = S::JS / ((S::VB + 15) / 16);      // MMAs of a chunk
#pragma unroll
                for (int g = 0; g < PER; g += 4) {                   // hi parts of four, then their lo parts
                    uint32_t av[4][4];
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        const int i = g + q4;
                        if constexpr (Q8) {
                            const uint32_t sel = i % 2 ? 0x7362u : 0x5140u;   // two elements of both tokens, element-major
                            e4m3x4_to_f16x2(__byte_perm(v[0][i / 2], v[1][i / 2], sel), av[q4][0], av[q4][1]);
                            e4m3x4_to_f16x2(__byte_perm(v[2][i / 2], v[3][i / 2], sel), av[q4][2], av[q4][3]);
                        } else {
                            av[q4][0] = __byte_perm(v[0][i], v[1][i], 0x5410);
                            av[q4][1] = __byte_perm(v[0][i], v[1][i], 0x7632);
                            av[q4][2] = __byte_perm(v[2][i], v[3][i], 0x5410);
                            av[q4][3] = __byte_perm(v[2][i], v[3][i], 0x7632);
                        }
                    }
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<Q8>(oacc[nt][c * PER + g + q4], av[q4][0], av[q4][1], av[q4][2], av[q4][3],
                                             part ? bl[nt][0] : bh[nt][0], part ? bl[nt][1] : bh[nt][1]);
                }
            }
        }
        __syncthreads();   // every warp is done with its ring: reuse it for the merge
        if (abort_flag) return;

        // ---- merge the warps' states per head ----
        const float oscale = Q8 ? exp2_whole(evref) : 1.f;
        float *mg = merge + warp * S::HEADS * S::MSTRIDE;
#pragma unroll
        for (int h = 0; h < S::HPT; ++h) {
            const int head = RHO ? 4 * h + t4 : 8 * (h / 2) + 2 * t4 + h % 2;
            float l = lsum[h], ab = asum[h];
#pragma unroll
            for (int off = 4; off < 32; off *= 2) {
                l += __shfl_xor_sync(0xffffffffu, l, off);
                ab += __shfl_xor_sync(0xffffffffu, ab, off);
            }
            float *row = mg + head * S::MSTRIDE;
            if (r == 0) {
                row[0] = mref[h];
                row[1] = l;
                row[2] = ab;
            }
            const int nt = RHO ? h : h / 2;
#pragma unroll
            for (int j = 0; j < S::JS; ++j) {
                // rows r and r + 8 of the product's step j are elements d and d + 1
                const int d = Q8 || S::VB == 16 ? (S::VB / S::EL) * r + 2 * j : 64 * (j / 4) + 8 * r + 2 * (j % 4);
                if constexpr (RHO) {
                    row[4 + d] = oacc[nt][j][0] * oscale;
                    row[4 + d + 1] = oacc[nt][j][2] * oscale;
                    row[4 + D + d] = oacc[nt][j][1] * (oscale * ASCALE);
                    row[4 + D + d + 1] = oacc[nt][j][3] * (oscale * ASCALE);
                } else {
                    row[4 + d] = oacc[nt][j][h % 2] * oscale;
                    row[4 + d + 1] = oacc[nt][j][2 + h % 2] * oscale;
                }
            }
        }
        __syncthreads();
        for (int idx = threadIdx.x; idx < nh * D; idx += WARPS * 32) {
            const int hh = idx / D, e = idx % D;
            float mu = MNONE;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) mu = fmaxf(mu, merge[(w * S::HEADS + hh) * S::MSTRIDE]);
            float l = 0.f, ab = 0.f, o = 0.f, m = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float *src = merge + (w * S::HEADS + hh) * S::MSTRIDE;
                const float f = fex2(src[0] - mu);    // 0 for a warp without a tile
                l = fmaf(f, src[1], l);
                o = fmaf(f, src[4 + e], o);
                if constexpr (RHO) {
                    ab = fmaf(f, src[2], ab);
                    m = fmaf(f, src[4 + D + e], m);
                }
            }
            const long bh = h0 + hh;
            if (nsplit == 1) {
                float out = 0.f;
                if (ntiles > 0) {
                    const float inv = 1.0f / l;
                    out = o * inv;
                    if constexpr (RHO) out -= m * inv - out * (ab * inv);
                }
                store_y<Tout>(y + bh * D + e, out);
                if (e == 0 && lse != nullptr) lse[bh] = ntiles > 0 ? (mu + log2f(l)) * LN2 : -INFINITY;
            } else {
                float *P = parts + ((size_t)bh * nsplit + split) * part_stride<D, RHO>();
                P[e] = o;
                if constexpr (RHO) P[D + e] = m;
            }
            if (e == 0 && hdr != nullptr) hdr[bh * nsplit + split] = make_float4(mu, l, ab, 0.f);
        }
        fence_proxy_async();   // the next unit's copies write where these stores and loads went
        __syncthreads();
    }
}

// One launch after the split kernel: blocks [0, combine_blocks) merge the splits
// of one (b, h) each and write y and lse; the others add the weights
// s = 2^(z - lse2) of ACC_TOKENS tokens of one (b, kvh) to the accumulator, summed
// over the KV head's query heads in head order (each token by one thread:
// the result does not depend on the schedule).
constexpr int FIN_THREADS = 256;
constexpr int ACC_TOKENS = 1024;

template <int D, bool RHO, int HEADS, typename Tout>
__global__ void __launch_bounds__(FIN_THREADS) k_decode_finish(
    const float *__restrict__ parts, const float4 *__restrict__ hdr, const float *__restrict__ zs,
    const int *__restrict__ seqlens, Tout *__restrict__ y, float *__restrict__ lse, float *__restrict__ wacc, int Hq,
    int Hkv, int htiles, int chunk, int nsplit, int Tcap, long combine_blocks, int acc_chunks) {
    constexpr int COLS = (RHO ? 2 : 1) * D / 4;               // float4 columns of a partial
    constexpr int GROUPS = FIN_THREADS / COLS;                // splits in flight
    __shared__ float4 red[GROUPS][COLS];
    __shared__ float2 redl[GROUPS];
    __shared__ float wred[FIN_THREADS / 32];
    __shared__ float slse[HEADS];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if ((long)blockIdx.x < combine_blocks) {
        const long bh = blockIdx.x;
        const int L = min(max(seqlens[bh / Hq], 0), Tcap);
        const int nv = (L + chunk - 1) / chunk;
        if (nv == 0) {
            for (int e = tid; e < D; e += FIN_THREADS) store_y<Tout>(y + bh * D + e, 0.f);
            if (lse != nullptr && tid == 0) lse[bh] = -INFINITY;
            return;
        }
        const float4 *H = hdr + bh * nsplit;
        float mu = -INFINITY;
        for (int s = tid; s < nv; s += FIN_THREADS) mu = fmaxf(mu, H[s].x);
#pragma unroll
        for (int off = 16; off > 0; off /= 2) mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, off));
        if (lane == 0) wred[warp] = mu;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < FIN_THREADS / 32; ++w) mu = fmaxf(mu, wred[w]);
        const int col = tid % COLS, grp = tid / COLS;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f, ab = 0.f;
        const float4 *P = reinterpret_cast<const float4 *>(parts) + (size_t)bh * nsplit * COLS + col;
#pragma unroll 4
        for (int s = grp; s < nv; s += GROUPS) {
            const float4 h = H[s];
            const float4 p = P[(size_t)s * COLS];
            const float w = fex2(h.x - mu);
            l = fmaf(w, h.y, l);
            ab = fmaf(w, h.z, ab);
            acc.x = fmaf(w, p.x, acc.x);
            acc.y = fmaf(w, p.y, acc.y);
            acc.z = fmaf(w, p.z, acc.z);
            acc.w = fmaf(w, p.w, acc.w);
        }
        red[grp][col] = acc;
        if (col == 0) redl[grp] = make_float2(l, ab);
        __syncthreads();
        l = ab = 0.f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            l += redl[g].x;
            ab += redl[g].y;
        }
        const float inv = 1.f / l;
        const float *R = reinterpret_cast<const float *>(red);
        for (int e = tid; e < D; e += FIN_THREADS) {
            float o = 0.f, m = 0.f;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                o += R[g * COLS * 4 + e];
                if constexpr (RHO) m += R[g * COLS * 4 + D + e];
            }
            float out = o * inv;
            if constexpr (RHO) out -= m * inv - out * (ab * inv);
            store_y<Tout>(y + bh * D + e, out);
        }
        if (lse != nullptr && tid == 0) lse[bh] = (mu + log2f(l)) * LN2;
        return;
    }
    // ---- accumulate ----
    const long ab_ = (long)blockIdx.x - combine_blocks;
    const int ck = (int)(ab_ % acc_chunks);
    const long bk = ab_ / acc_chunks;                          // b * Hkv + kvh
    const int b = (int)(bk / Hkv), kvh = (int)(bk % Hkv), group = Hq / Hkv;
    const int L = min(max(seqlens[b], 0), Tcap);
    const int t0 = ck * ACC_TOKENS;
    if (t0 >= L) return;
    const int nv = (L + chunk - 1) / chunk;
    constexpr int PER = ACC_TOKENS / FIN_THREADS;
    float sum[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) sum[k] = 0.f;
    for (int ht = 0; ht < htiles; ++ht) {
        const int nh = min(HEADS, group - ht * HEADS);
        __syncthreads();
        for (int h = warp; h < nh; h += FIN_THREADS / 32) {
            const float4 *H = hdr + ((long)b * Hq + (long)kvh * group + ht * HEADS + h) * nsplit;
            float mu = -INFINITY, l = 0.f;
            for (int s = lane; s < nv; s += 32) mu = fmaxf(mu, H[s].x);
#pragma unroll
            for (int off = 16; off > 0; off /= 2) mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, off));
            for (int s = lane; s < nv; s += 32) l += fex2(H[s].x - mu) * H[s].y;
#pragma unroll
            for (int off = 16; off > 0; off /= 2) l += __shfl_xor_sync(0xffffffffu, l, off);
            if (lane == 0) slse[h] = mu + log2f(l);
        }
        __syncthreads();
        const float *Z = zs + (((size_t)bk * htiles + ht) * (size_t)Tcap) * HEADS;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int t = t0 + tid + k * FIN_THREADS;
            if (t >= L) continue;
            const float4 *zr = reinterpret_cast<const float4 *>(Z + (size_t)t * HEADS);
#pragma unroll
            for (int c = 0; c < HEADS / 4; ++c) {
                if (4 * c >= nh) break;
                const float4 zv = zr[c];
                sum[k] += fex2(zv.x - slse[4 * c]);
                if (4 * c + 1 < nh) sum[k] += fex2(zv.y - slse[4 * c + 1]);
                if (4 * c + 2 < nh) sum[k] += fex2(zv.z - slse[4 * c + 2]);
                if (4 * c + 3 < nh) sum[k] += fex2(zv.w - slse[4 * c + 3]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int t = t0 + tid + k * FIN_THREADS;
        if (t < L) wacc[(size_t)bk * Tcap + t] += sum[k];
    }
}

// heads of a unit for a group of query heads
template <bool RHO> int heads_for(int group) { return RHO ? (group <= 4 ? 4 : 8) : 8; }

template <int D, bool Q8, bool RHO, int NT, typename Tout>
cudaError_t launch_t(const DecodeCacheArgs &A, const DecodePlan &p, void *ws, const DeviceCtl &ctl, cudaStream_t s) {
    using S = Shape<D, Q8, RHO, NT>;
    const int htiles = (A.pg.group + S::HEADS - 1) / S::HEADS;
    const int Tcap = A.pg.max_pages << A.pg.pshift;
    const long BH = (long)A.B * A.Hq;
    const DecodeCacheScratch sc = decode_cache_scratch(A, p);
    char *base = static_cast<char *>(ws);
    float *parts = sc.parts ? reinterpret_cast<float *>(base) : nullptr;
    float4 *hdr = sc.hdr ? reinterpret_cast<float4 *>(base + sc.parts) : nullptr;
    float *zs = sc.zs ? reinterpret_cast<float *>(base + sc.parts + sc.hdr) : nullptr;
    const long per_split = (long)A.B * A.pg.Hkv * htiles;
    const long units = per_split * p.nsplit;
    static std::atomic<unsigned long long> limit_set{0};
    if (cudaError_t e = ensure_smem_limit(k_decode_cache<D, Q8, RHO, NT, Tout>, S::SMEM, limit_set)) return e;
    k_decode_cache<D, Q8, RHO, NT, Tout><<<(unsigned)(units < 0x7fffffffL ? units : 0x7fffffffL), WARPS * 32, S::SMEM, s>>>(
        (const __nv_bfloat16 *)A.q, (const __nv_bfloat16 *)A.rho, (const uint8_t *)A.kpages, (const uint8_t *)A.vpages,
        A.kexp, A.vexp, A.seqlens, (Tout *)A.y, A.lse, A.Hq, p.chunk, p.nsplit, per_split, htiles, A.pg, parts, hdr, zs,
        ctl);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (p.nsplit == 1 && A.wacc == nullptr)) return e;
    const long combine = p.nsplit > 1 ? BH : 0;
    const int acc_chunks = A.wacc ? (Tcap + ACC_TOKENS - 1) / ACC_TOKENS : 0;
    const long blocks = combine + (long)A.B * A.pg.Hkv * acc_chunks;
    k_decode_finish<D, RHO, S::HEADS, Tout><<<(unsigned)blocks, FIN_THREADS, 0, s>>>(
        parts, hdr, zs, A.seqlens, (Tout *)A.y, A.lse, A.wacc, A.Hq, A.pg.Hkv, htiles, p.chunk, p.nsplit, Tcap, combine,
        acc_chunks);
    return cudaGetLastError();
}

template <int D, bool Q8, typename Tout>
cudaError_t launch_d(const DecodeCacheArgs &A, const DecodePlan &p, void *ws, const DeviceCtl &ctl, cudaStream_t s) {
    if (A.rho == nullptr) return launch_t<D, Q8, false, 1, Tout>(A, p, ws, ctl, s);
    if (A.pg.group <= 4) return launch_t<D, Q8, true, 1, Tout>(A, p, ws, ctl, s);
    return launch_t<D, Q8, true, 2, Tout>(A, p, ws, ctl, s);
}

}  // namespace

int decode_cache_heads(bool with_rho, int group) { return with_rho ? heads_for<true>(group) : heads_for<false>(group); }

DecodeCacheScratch decode_cache_scratch(const DecodeCacheArgs &A, const DecodePlan &p) {
    const size_t up = 255;
    const size_t BHS = (size_t)A.B * A.Hq * p.nsplit;
    const int heads = decode_cache_heads(A.rho != nullptr, A.pg.group);
    const size_t htiles = (A.pg.group + heads - 1) / heads;
    DecodeCacheScratch s;
    s.parts = p.nsplit > 1 ? (BHS * (A.rho ? 2 : 1) * A.d * sizeof(float) + up) & ~up : 0;
    s.hdr = p.nsplit > 1 || A.wacc ? (BHS * 16 + up) & ~up : 0;
    s.zs = A.wacc ? (size_t)A.B * A.pg.Hkv * htiles * ((size_t)A.pg.max_pages << A.pg.pshift) * heads * sizeof(float) : 0;
    return s;
}

cudaError_t launch_decode_cache(const DecodeCacheArgs &A, const DecodePlan &p, void *ws, const DeviceCtl &ctl,
                                cudaStream_t s) {
    const bool f32 = A.out_dtype == PARALLAX_F32;
    if (A.d == 64) {
        if (A.kexp)
            return f32 ? launch_d<64, true, float>(A, p, ws, ctl, s) : launch_d<64, true, __nv_bfloat16>(A, p, ws, ctl, s);
        return f32 ? launch_d<64, false, float>(A, p, ws, ctl, s) : launch_d<64, false, __nv_bfloat16>(A, p, ws, ctl, s);
    }
    if (A.kexp)
        return f32 ? launch_d<128, true, float>(A, p, ws, ctl, s) : launch_d<128, true, __nv_bfloat16>(A, p, ws, ctl, s);
    return f32 ? launch_d<128, false, float>(A, p, ws, ctl, s) : launch_d<128, false, __nv_bfloat16>(A, p, ws, ctl, s);
}

}  // namespace plx
