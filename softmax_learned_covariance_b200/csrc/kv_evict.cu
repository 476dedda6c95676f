// kv_evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// Per sequence and KV head, of L tokens n = min(L, budget) stay: the newest
// min(recent, n) and, of the others, the heaviest by the accumulator (equal
// weights: the lower position; NaN counts as -inf).  They keep their order and
// go to positions 0 .. n-1 of the pages a second table names; the source pages
// are only read.
//
// Two launches.  k_evict_select finds the weight of the last kept token by a
// radix select over order-preserving integer keys and writes the kept
// positions in order; k_evict_move copies the rows, one warp per 16-row
// destination block.  An e4m3 destination block takes the largest exponent of
// its rows' source blocks and the rows of smaller ones are moved to it (exact
// until subnormal).
#include "cache_common.cuh"

namespace plx {
namespace {

constexpr int SEL_THREADS = 1024;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int MOVE_WARPS = 4;

// Weights as integers in the same order: -0 and +0 are equal, NaN is -inf.
__device__ __forceinline__ uint32_t order_key(float x) {
    uint32_t u = __float_as_uint(x);
    if ((u & 0x7fffffffu) > 0x7f800000u) u = 0xff800000u;
    if (u == 0x80000000u) u = 0u;
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Exclusive sum over the block of one value per thread; `total` gets the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *wsum, uint32_t &total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += o;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    uint32_t s = lane < SEL_WARPS ? wsum[lane] : 0u;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
    return x - v + (warp > 0 ? before : 0u);
}

__global__ void __launch_bounds__(SEL_THREADS) k_evict_select(KvEvictArgs A) {
    __shared__ uint32_t hist[2048];
    __shared__ uint32_t wsum[32];
    __shared__ uint32_t pick, above;
    const int tid = threadIdx.x;
    const long bk = blockIdx.x;
    const int b = (int)(bk / A.pg.Hkv);
    const int cap = A.pg.max_pages << A.pg.pshift;
    const size_t ncap = (size_t)A.new_max_pages << A.pg.pshift;
    const int L = min(max(A.seqlens[b], 0), cap);
    const int n = min(L, A.budget), tail = min(A.recent, n);
    const int C = L - tail, need = n - tail;           // `need` of the first C, then the last `tail`
    if (bk % A.pg.Hkv == 0 && tid == 0) A.new_seqlens[b] = n;
    const float *w = A.wacc + (size_t)bk * cap;
    int *kept = A.kept + (size_t)bk * A.budget;
    float *nw = A.new_wacc ? A.new_wacc + bk * ncap : nullptr;

    uint32_t prefix = 0, mask = 0, ties = 0;           // the need-th largest key, found from the top bits down
    if (need > 0 && need < C) {
        uint32_t left = (uint32_t)need;                // how many of the keys that match `prefix` are wanted
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
            const int bits = pass == 2 ? 10 : 11;
            for (int i = tid; i < 2048; i += SEL_THREADS) hist[i] = 0u;
            __syncthreads();
            for (int t = tid; t < C; t += SEL_THREADS) {
                const uint32_t k = order_key(w[t]);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
            }
            __syncthreads();
            // thread i owns the bins 2047 - 2i and 2046 - 2i: an exclusive sum from the largest bin down
            const uint32_t h0 = hist[2047 - 2 * tid], h1 = hist[2046 - 2 * tid];
            uint32_t total;
            const uint32_t before = block_scan(h0 + h1, wsum, total);
            if (before < left && left <= before + h0 + h1) {
                const bool first = left <= before + h0;
                pick = (uint32_t)(first ? 2047 - 2 * tid : 2046 - 2 * tid);
                above = first ? before : before + h0;
            }
            __syncthreads();
            prefix |= pick << shift;
            mask |= ((1u << bits) - 1u) << shift;
            left -= above;
            __syncthreads();
        }
        ties = left;                                   // this many of the tokens whose key is `prefix`, in order
    }
    // ---- kept positions in order ----
    uint32_t done = 0, tied = 0;                       // kept so far; of them equal to the last kept key
    if (need > 0) {
        const bool all = need == C;
        for (int base = 0; base < C; base += SEL_THREADS) {
            const int t = base + tid;
            const float x = t < C ? w[t] : 0.f;
            const uint32_t k = order_key(x);
            const bool gt = t < C && (all || k > prefix), eq = t < C && !all && k == prefix;
            // two counts in one sum: larger keys low, equal keys high (at most 1024 each)
            uint32_t total;
            const uint32_t sc = block_scan((gt ? 1u : 0u) | (eq ? 1u << 16 : 0u), wsum, total);
            const uint32_t eq_before = tied + (sc >> 16);
            const bool keep = gt || (eq && eq_before < ties);
            if (keep) {
                const uint32_t at = done + (sc & 0xffffu) + min(eq_before, ties) - min(tied, ties);
                kept[at] = t;
                if (nw) nw[at] = x;
            }
            const uint32_t eq_now = min(tied + (total >> 16), ties) - min(tied, ties);
            done += (total & 0xffffu) + eq_now;
            tied += total >> 16;
        }
    }
    for (int i = tid; i < tail; i += SEL_THREADS) {
        kept[need + i] = C + i;
        if (nw) nw[need + i] = w[C + i];
    }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(MOVE_WARPS * 32) k_evict_move(KvEvictArgs A, long units, int nblocks, int *__restrict__ err) {
    constexpr int ROW = D * (Q8 ? 1 : 2);
    constexpr int CH = ROW / 16;             // 16-byte chunks of a row
    constexpr int RPI = 32 / CH;             // rows per warp access
    constexpr int LOADS = KV_BLOCK / RPI;
    const int lane = threadIdx.x % 32;
    const long u = (long)blockIdx.x * MOVE_WARPS + threadIdx.x / 32;
    if (u >= units) return;
    const bool is_v = u & 1;
    const int blk = (int)((u >> 1) % nblocks);
    const long bk = (u >> 1) / nblocks;
    const int b = (int)(bk / A.pg.Hkv), kvh = (int)(bk % A.pg.Hkv);
    const int ps = 1 << A.pg.pshift;
    const int L = min(max(A.seqlens[b], 0), A.pg.max_pages << A.pg.pshift);
    const int n = min(L, A.budget);
    const int i0 = blk * KV_BLOCK;
    if (i0 >= n) return;
    const int rows = min(KV_BLOCK, n - i0);
    const int did = A.new_table[(size_t)b * A.new_max_pages + (i0 >> A.pg.pshift)];
    if ((unsigned)did >= (unsigned)A.pg.num_pages) {
        if (lane == 0) atomicExch(err, PARALLAX_ERR_DEVICE_INDEX);
        return;
    }
    uint8_t *pages = static_cast<uint8_t *>(is_v ? A.vpages : A.kpages);
    signed char *exps = is_v ? A.vexp : A.kexp;
    // lane i < rows: where row i comes from (-1: a page id out of range, the row is zero)
    long long from = -1;
    int e = KV_EMIN;
    if (lane < rows) {
        const int t = A.kept[(size_t)bk * A.budget + i0 + lane];
        const int id = A.pg.table[(size_t)b * A.pg.max_pages + (t >> A.pg.pshift)];
        if ((unsigned)id < (unsigned)A.pg.num_pages) {
            const size_t slab = (size_t)id * A.pg.Hkv + kvh;
            from = (long long)(slab * ps + (t & (ps - 1)));
            if constexpr (Q8) e = exps[slab * (ps / KV_BLOCK) + (t & (ps - 1)) / KV_BLOCK];
        } else {
            atomicExch(err, PARALLAX_ERR_DEVICE_INDEX);
        }
    }
    const size_t dslab = (size_t)did * A.pg.Hkv + kvh;
    const int drow = i0 & (ps - 1);
    uint8_t *dst = pages + (dslab * ps + drow) * ROW;
    const int ch = lane % CH, rr = lane / CH;
    uint4 w[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = i * RPI + rr;
        const long long f = __shfl_sync(0xffffffffu, from, row);
        w[i] = f >= 0 ? *reinterpret_cast<const uint4 *>(pages + f * ROW + ch * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (Q8) {
        int emax = e;
#pragma unroll
        for (int off = 16; off > 0; off /= 2) emax = max(emax, __shfl_xor_sync(0xffffffffu, emax, off));
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int es = __shfl_sync(0xffffffffu, e, i * RPI + rr);
            if (es < emax) w[i] = e4m3_shift_down(w[i], emax - es);
        }
        if (lane == 0) exps[dslab * (ps / KV_BLOCK) + drow / KV_BLOCK] = (signed char)emax;
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = i * RPI + rr;
        if (row < rows) *reinterpret_cast<uint4 *>(dst + row * ROW + ch * 16) = w[i];
    }
}

template <int D, bool Q8> cudaError_t launch_move(const KvEvictArgs &A, int *err, cudaStream_t s) {
    const int nblocks = (A.budget + KV_BLOCK - 1) / KV_BLOCK;
    const long units = (long)A.B * A.pg.Hkv * nblocks * 2;
    k_evict_move<D, Q8><<<(unsigned)((units + MOVE_WARPS - 1) / MOVE_WARPS), MOVE_WARPS * 32, 0, s>>>(A, units, nblocks, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_evict(const KvEvictArgs &A, const DeviceCtl &ctl, cudaStream_t s) {
    k_evict_select<<<(unsigned)((long)A.B * A.pg.Hkv), SEL_THREADS, 0, s>>>(A);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (A.d == 64) return A.kexp ? launch_move<64, true>(A, ctl.err, s) : launch_move<64, false>(A, ctl.err, s);
    return A.kexp ? launch_move<128, true>(A, ctl.err, s) : launch_move<128, false>(A, ctl.err, s);
}

}  // namespace plx
