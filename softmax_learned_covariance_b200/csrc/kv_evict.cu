// kv_evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// Per sequence and KV head, of L tokens n = min(L, budget) stay: the newest
// min(recent, n) and, of the others, the heaviest by the accumulator (equal
// weights: the lower position; NaN counts as -inf).  They keep their order and
// go to positions 0 .. n-1 of the pages a second table names; the source pages
// are only read.
//
// Two launches.  k_evict_select finds the weight of the last kept token by a
// radix select over order-preserving integer keys (three digits of 11, 11 and 10
// bits) and writes the kept positions in order: a cluster of CTAs per head, which add
// the bins they hit to the first one's histogram (reading all histograms in all
// CTAs took the cluster's shared memories 2 us a digit); a CTA whose share is at most
// SEL_TILE tokens reads its weights once and keeps the keys in registers.
// k_evict_move copies the rows, one warp per 16-row destination block (K and V).  An e4m3
// destination block takes the largest exponent of its rows' source blocks and the
// rows of smaller ones are moved to it (exact until subnormal).
//
// Measured: 64 sequences of 3000-4096, 8 heads, 2048 kept, e4m3: 108 us a call; the
// move 86 (0.55 GB read and written, 6.3 TB/s of 6.57), the selection 18, bound by
// instruction issue and barriers.  One sequence of 32768, 8 heads, 4096 kept, bf16:
// 20 us, of them 12.5 the selection (41 with one CTA per head), latency.
#include <cooperative_groups.h>

#include "cache_common.cuh"

namespace plx {
namespace {

constexpr int SEL_THREADS = 512;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_ITEMS = 8;                            // tokens of a thread at a time
constexpr int SEL_TILE = SEL_THREADS * SEL_ITEMS;
constexpr int BINS = 2048, OWN = BINS / SEL_THREADS;    // bins, and those a thread sums
constexpr int MOVE_WARPS = 4;
static_assert(3 * BINS >= SEL_TILE, "the kept positions of a tile reuse the histograms");

// Weights as integers in the same order: -0 and +0 are equal, NaN is -inf.  The
// smallest key is 0x007fffff; 0 stands for no token.
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

template <bool CLUSTER>
__global__ void __launch_bounds__(SEL_THREADS, CLUSTER ? 2 : 4) k_evict_select(KvEvictArgs A, int ctas) {
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int cluster_size = CLUSTER ? ctas : 1;
    auto sync = [&] {
        if constexpr (CLUSTER)
            cluster.sync();
        else
            __syncthreads();
    };
    __shared__ __align__(16) uint32_t hist[3][BINS];
    __shared__ uint32_t wsum[32];
    __shared__ uint32_t found[3], mine[2];             // a digit, the keys above it and with it; this CTA's counts
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, rank = CLUSTER ? (int)(blockIdx.x % (unsigned)cluster_size) : 0;
    const unsigned bk = blockIdx.x / (unsigned)cluster_size;
    const int b = (int)(bk / (unsigned)A.pg.Hkv);
    const int cap = A.pg.max_pages << A.pg.pshift;
    const size_t ncap = (size_t)A.new_max_pages << A.pg.pshift;
    const int L = min(max(A.seqlens[b], 0), cap);
    const int n = min(L, A.budget), tail = min(A.recent, n);
    const int C = L - tail, need = n - tail;           // `need` of the first C, then the last `tail`
    if (bk == (unsigned)b * A.pg.Hkv && rank == 0 && tid == 0) A.new_seqlens[b] = n;
    const float *w = A.wacc + (size_t)bk * cap;
    int *kept = A.kept + (size_t)bk * A.budget;
    float *nw = A.new_wacc ? A.new_wacc + bk * ncap : nullptr;
    auto keep_tail = [&] {
        for (int i = rank * SEL_THREADS + tid; i < tail; i += cluster_size * SEL_THREADS) {
            kept[need + i] = C + i;
            if (nw) nw[need + i] = w[C + i];
        }
    };
    if (need == 0) {                                   // the whole cluster
        keep_tail();
        return;
    }
    // this CTA's candidates [begin, end)
    const int share = ((C + cluster_size - 1) / cluster_size + 3) & ~3;
    const int begin = min(rank * share, C), end = min(begin + share, C);
    const bool all = need == C, once = share <= SEL_TILE;

    uint32_t key[SEL_ITEMS];
    auto load = [&](int base) {                        // tokens base + SEL_ITEMS tid ..
#pragma unroll
        for (int v = 0; v < SEL_ITEMS; v += 4) {
            const int t = base + SEL_ITEMS * tid + v;
            const float4 f = t < end ? *reinterpret_cast<const float4 *>(w + t) : make_float4(0.f, 0.f, 0.f, 0.f);
            key[v] = t < end ? order_key(f.x) : 0u;
            key[v + 1] = t + 1 < end ? order_key(f.y) : 0u;
            key[v + 2] = t + 2 < end ? order_key(f.z) : 0u;
            key[v + 3] = t + 3 < end ? order_key(f.w) : 0u;
        }
    };
    if (once) load(begin);
    uint32_t prefix = 0, mask = 0, ties = 0;           // the need-th largest key, found from the top bits down
    if (!all) {
        for (int i = tid; i < 3 * BINS / 4; i += SEL_THREADS) reinterpret_cast<uint4 *>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
        sync();                                        // zero before any CTA of the cluster adds to it
        uint32_t left = (uint32_t)need;                // how many of the keys that match `prefix` are wanted
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
            const uint32_t digit = pass == 2 ? 1023u : 2047u;
            for (int base = begin; base < end; base += SEL_TILE) {
                if (!once) load(base);
#pragma unroll
                for (int i = 0; i < SEL_ITEMS; ++i) {
                    const uint32_t k = key[i];
                    if ((k & mask) == prefix && k != 0u) atomicAdd(&hist[pass][(k >> shift) & digit], 1u);
                }
            }
            __syncthreads();                           // this CTA's histogram of the digit is complete
            // thread i owns the OWN bins below BINS - OWN i
            const int top = BINS - OWN * (tid + 1);
            uint32_t h[OWN];
            auto read = [&] {
#pragma unroll
                for (int i = 0; i < OWN; i += 4) {
                    const uint4 o = *reinterpret_cast<const uint4 *>(&hist[pass][top + i]);
                    h[i] = o.x;
                    h[i + 1] = o.y;
                    h[i + 2] = o.z;
                    h[i + 3] = o.w;
                }
            };
            read();
            if constexpr (CLUSTER) {
                if (rank != 0) {
                    uint32_t *first = cluster.map_shared_rank(&hist[pass][top], 0);
#pragma unroll
                    for (int i = 0; i < OWN; ++i)
                        if (h[i]) atomicAdd(first + i, h[i]);
                }
                cluster.sync();
                read();
            }
            if (rank == 0) {
                // an exclusive sum from the largest bin down finds the bin of the last wanted key
                uint32_t total, own = 0;
#pragma unroll
                for (int i = 0; i < OWN; ++i) own += h[i];
                uint32_t before = block_scan(own, wsum, total);
                if (before < left && left <= before + own) {
                    int i = OWN - 1;
                    for (; i > 0 && before + hist[pass][top + i] < left; --i) before += hist[pass][top + i];
                    for (int q = 0; q < cluster_size; ++q) {
                        uint32_t *to = CLUSTER ? cluster.map_shared_rank(found, q) : found;
                        to[0] = (uint32_t)(top + i);
                        to[1] = before;
                        to[2] = hist[pass][top + i];
                    }
                }
            }
            sync();
            prefix |= found[0] << shift;
            mask |= digit << shift;
            left -= found[1];
            if (found[2] == left) {
                // every key with this prefix is wanted (after two digits nearly always: the
                // one key there): all that are larger than the largest key below it
                prefix -= 1u;
                left = 0;
                break;
            }
        }
        ties = left;                                   // this many of the tokens whose key is `prefix`, in order
    }
    // Larger keys (low half: at most SEL_TILE of a CTA) and equal ones (high half) of a
    // thread's tokens; when all are kept, prefix and ties are 0.
    auto count = [&] {
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < SEL_ITEMS; ++i) c += key[i] > prefix ? 1u : (key[i] == prefix ? 1u << 16 : 0u);
        return c;
    };
    uint32_t larger = 0, tied = 0;                     // before this CTA's tokens, then before the tile's
    if constexpr (CLUSTER) {
        uint32_t g = 0, e = 0;
        for (int base = begin; base < end; base += SEL_TILE) {
            if (!once) load(base);
            uint32_t total;
            block_scan(count(), wsum, total);
            g += total & 0xffffu;
            e += total >> 16;
        }
        if (tid == 0) {
            mine[0] = g;
            mine[1] = e;
        }
        cluster.sync();
        for (int q = 0; q < rank; ++q) {
            const uint32_t *theirs = cluster.map_shared_rank(&mine[0], q);
            larger += theirs[0];
            tied += theirs[1];
        }
    }
    // ---- kept positions in order, through shared memory, so that whole lines are stored
    // (one by one: 20 against 18.5 us for 512 heads of 4096) ----
    int *staged = reinterpret_cast<int *>(hist);       // SEL_TILE of them; the histograms are done
    for (int base = begin; base < end; base += SEL_TILE) {
        if (!once) load(base);
        uint32_t total;
        const uint32_t sc = block_scan(count(), wsum, total);
        const uint32_t from = larger + min(tied, ties);
        uint32_t g = larger + (sc & 0xffffu), e = tied + (sc >> 16);
#pragma unroll
        for (int i = 0; i < SEL_ITEMS; ++i) {
            const bool gt = key[i] > prefix, eq = key[i] == prefix;
            if (gt || (eq && e < ties)) staged[g + min(e, ties) - from] = base + SEL_ITEMS * tid + i;
            g += gt;
            e += eq;
        }
        larger += total & 0xffffu;
        tied += total >> 16;
        __syncthreads();
        const uint32_t n_here = larger + min(tied, ties) - from;
#pragma unroll 4
        for (uint32_t i = tid; i < n_here; i += SEL_THREADS) kept[from + i] = staged[i];
        if (nw) {
#pragma unroll 4
            for (uint32_t i = tid; i < n_here; i += SEL_THREADS) nw[from + i] = w[staged[i]];
        }
        __syncthreads();
    }
    keep_tail();
    if constexpr (CLUSTER) cluster.sync();             // no CTA leaves while its counts are read
}

template <int D, bool Q8>
__global__ void __launch_bounds__(MOVE_WARPS * 32) k_evict_move(KvEvictArgs A, unsigned units, unsigned nblocks, int *__restrict__ err) {
    constexpr int ROW = D * (Q8 ? 1 : 2);
    constexpr int CH = ROW / 16;             // 16-byte chunks of a row
    constexpr int RPI = 32 / CH;             // rows per warp access
    constexpr int LOADS = KV_BLOCK / RPI;
    const int lane = threadIdx.x % 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const unsigned u = blockIdx.x * MOVE_WARPS + threadIdx.x / 32;
    if (u >= units) return;
    const int blk = (int)(u % nblocks);
    const unsigned bk = u / nblocks;
    const int b = (int)(bk / (unsigned)A.pg.Hkv), kvh = (int)(bk % (unsigned)A.pg.Hkv);
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
    // lane i < rows: where row i comes from (-1: a page id out of range, the row is zero)
    long long from = -1;
    int e[2] = {KV_EMIN, KV_EMIN};
    if (lane < rows) {
        const int t = A.kept[(size_t)bk * A.budget + i0 + lane];
        const int id = A.pg.table[(size_t)b * A.pg.max_pages + (t >> A.pg.pshift)];
        if ((unsigned)id < (unsigned)A.pg.num_pages) {
            const size_t slab = (size_t)id * A.pg.Hkv + kvh;
            from = (long long)(slab * ps + (t & (ps - 1)));
            if constexpr (Q8) {
                e[0] = A.kexp[slab * (ps / KV_BLOCK) + (t & (ps - 1)) / KV_BLOCK];
                e[1] = A.vexp[slab * (ps / KV_BLOCK) + (t & (ps - 1)) / KV_BLOCK];
            }
        } else {
            atomicExch(err, PARALLAX_ERR_DEVICE_INDEX);
        }
    }
    const size_t dslab = (size_t)did * A.pg.Hkv + kvh;
    const int drow = i0 & (ps - 1);
    const int ch = lane % CH, rr = lane / CH;
    uint8_t *const pages[2] = {static_cast<uint8_t *>(A.kpages), static_cast<uint8_t *>(A.vpages)};
    uint4 w[2][LOADS];                                         // K and V rows: all loads before the first store
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const long long f = __shfl_sync(0xffffffffu, from, i * RPI + rr);
#pragma unroll
        for (int x = 0; x < 2; ++x)
            w[x][i] = f >= 0 ? *reinterpret_cast<const uint4 *>(pages[x] + f * ROW + ch * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if constexpr (Q8) {
            int emax = e[x];
#pragma unroll
            for (int off = 16; off > 0; off /= 2) emax = max(emax, __shfl_xor_sync(0xffffffffu, emax, off));
            // in most blocks all rows share an exponent or most do; a row below it is moved to it
            if (__any_sync(0xffffffffu, lane < rows && e[x] != emax)) {
#pragma unroll
                for (int i = 0; i < LOADS; ++i) {
                    const int es = __shfl_sync(0xffffffffu, e[x], i * RPI + rr);
                    if (es < emax) w[x][i] = e4m3_shift_down(w[x][i], emax - es);
                }
            }
            if (lane == 0) (x ? A.vexp : A.kexp)[dslab * (ps / KV_BLOCK) + drow / KV_BLOCK] = (signed char)emax;
        }
        uint8_t *dst = pages[x] + (dslab * ps + drow) * ROW;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int row = i * RPI + rr;
            if (row < rows) *reinterpret_cast<uint4 *>(dst + row * ROW + ch * 16) = w[x][i];
        }
    }
}

// The select, or with `dependent` the move as its programmatic dependent.
template <typename... P, typename... V>
cudaError_t launch_ex(void (*k)(P...), unsigned grid, unsigned threads, int cluster, bool dependent, cudaStream_t s,
                      V... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    if (dependent) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
    } else {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

template <int D, bool Q8> cudaError_t launch_move(const KvEvictArgs &A, int *err, cudaStream_t s) {
    const unsigned nblocks = (unsigned)(A.budget + KV_BLOCK - 1) / KV_BLOCK;
    const unsigned units = (unsigned)A.B * A.pg.Hkv * nblocks;      // below 2^31 (checked at entry)
    return launch_ex(k_evict_move<D, Q8>, (units + MOVE_WARPS - 1) / MOVE_WARPS, MOVE_WARPS * 32, 1, true, s,
                     A, units, nblocks, err);
}

}  // namespace

cudaError_t launch_kv_evict(const KvEvictArgs &A, int sm_count, const DeviceCtl &ctl, cudaStream_t s) {
    // up to 8 CTAs per head (the portable cluster size) while a CTA's share is more than
    // it keeps in registers and the heads alone do not fill the machine
    const long heads = (long)A.B * A.pg.Hkv;
    const int cap = A.pg.max_pages << A.pg.pshift;
    int cl = 1;
    while (cl < 8 && cap > cl * SEL_TILE && heads * cl < 2 * sm_count) cl *= 2;
    cudaError_t e = cl > 1 ? launch_ex(k_evict_select<true>, (unsigned)(heads * cl), SEL_THREADS, cl, false, s, A, cl)
                           : launch_ex(k_evict_select<false>, (unsigned)heads, SEL_THREADS, 1, false, s, A, 1);
    if (e != cudaSuccess) return e;
    if (A.d == 64) return A.kexp ? launch_move<64, true>(A, ctl.err, s) : launch_move<64, false>(A, ctl.err, s);
    return A.kexp ? launch_move<128, true>(A, ctl.err, s) : launch_move<128, false>(A, ctl.err, s);
}

}  // namespace plx
