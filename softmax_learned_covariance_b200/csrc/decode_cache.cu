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
// Each warp streams its own tiles of 32 tokens (16 of 256-byte rows) through a ring
// in shared memory that TMA fills, one box of 16 rows each for K and V (two for
// 256-byte rows).  The order of the contracted index is free as long as both
// operands agree, so a thread reads whole 16-byte chunks and uses them as its part
// of the fragments (K: chunks of its own two tokens; V: the same chunk of its four
// tokens): no ldmatrix, and no barrier beyond the warp's own mbarriers.  The order
// of the tokens is free too; with the hardware's swizzle it is chosen so that no
// read has a bank conflict (row_of).
//
// Bound by the loads, and how they are issued decides their rate (B=64, 16 heads of
// their own, 4096 tokens, d = 128, 1.07 GB; loads alone, merge launch included):
// 16-byte cp.async in fragment order 205 us, in row order 196 us, TMA 167 us.  The
// call takes 175-180 us, the kernel 166-172 (6.2-6.45 TB/s); B=16, 16 heads, 16384-32768
// tokens 257-265 us (6.1-6.3 TB/s of 6.57).  CTAs of equal ranges (decode_sched.h) end up to 20 %
// apart, but the memory is saturated until the last one does: ranges taken from a
// counter gained nothing.
//
// Numerics.  e4m3 codes are exact in fp16; q and rho are brought to fp16 by a
// power of two per vector (exact down to 2^-22 of the vector's largest
// element); the block exponents multiply z and a in fp32.  The weights of O and M
// are carried as two 16-bit parts.  For a bf16 cache, whose V needs no conversion,
// these are bf16: 2^-16 of any weight.  For an e4m3 cache they are fp16, 2^-21 with
// a smallest step of 2^-24, so what they are held against decides what is lost: per
// head, O's weights p 2^ve (ve: V's block exponent) against the largest so far, and
// M's, p |a| 2^ve, against their own; the largest is 2^10 to 2^15 in fp16.  What a
// token contributes is then off by 2^-35 of the largest contribution at most, which
// the fp32 sums lose as well.  (Held against the largest weight and the largest
// exponent, wherever each was met, a large V or a without weight cost every other
// token its bits.  The two references cost at most 1 % of the cases above,
// 4 % where two n-tiles meet a new item every few tiles.)  l and abar sum the fp32
// weights.
#include <math.h>

#include <type_traits>

#include "cache_common.cuh"
#include "decode_sched.h"
#include "sm100.cuh"

namespace plx {
namespace {

constexpr int WARPS = 4;
constexpr float MNONE = -1e30f;     // reference of a row that has seen no score
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
// A head's references move when a weight exceeds one by 2^4 (HEADROOM); fp16 weights of
// O and M are 2^WSHIFT at their reference, so 2^15 at most.
constexpr float HEADROOM = 16.f;
constexpr int WSHIFT = 11;

__device__ __forceinline__ float fex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// log2 of a power of two
__device__ __forceinline__ int whole_log2(float x) { return (__float_as_int(x) >> 23) - 127; }
// v 2^e for e in [-250, 250]
__device__ __forceinline__ float scaled(float v, int e) {
    const int half = e >> 1;
    return v * exp2_whole(half) * exp2_whole(e - half);
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

__device__ __forceinline__ void store_y2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
__device__ __forceinline__ void store_y2(__nv_bfloat16 *p, float a, float b) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}

constexpr int BAD = 1 << 16;     // a part's page id is out of range
// Exponents (-128, -128) of a part that is not there: below any other, so that it
// never sets the exponent O and M are held at.
constexpr int NO_EXPONENTS = 0x8080;

// Token of row i < 8 of the products' 16-row operand (row i + 8: the token + 8).
// A shared-memory phase is 8 threads of 16 bytes, rows 2 m and 2 m + 1 by four chunks
// of K, or chunks 2 m and 2 m + 1 by the rows 0, 2, 4, 6 or 1, 3, 5, 7 of V; each has
// to hit all 8 chunk columns once.  128-byte rows are swizzled by row & 7, 64-byte
// rows (two to a line; a V phase is 16 threads of 8 bytes) by (row >> 1) & 3.
template <int RB> __device__ __forceinline__ constexpr int row_of(int i) {
    if (RB == 64) return (i & 4) | ((i & 1) ? 3 - ((i >> 1) & 1) : (i >> 1) & 1);      // 0 3 1 2 4 7 5 6
    return (i & 1) ? i ^ 4 : i;                                                         // 0 5 2 7 4 1 6 3
}
// byte of 16-byte chunk c of row `row` of a swizzled box
template <int RB> __device__ __forceinline__ constexpr int chunk_at(int row, int c) {
    return row * RB + ((c ^ (RB == 64 ? (row >> 1) & 3 : row & 7)) << 4);
}

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
    static constexpr int RB = ROW < 128 ? ROW : 128;     // bytes of a box row (and of its swizzle)
    static constexpr int BOXES = ROW / RB;               // boxes of a K or V tile
    static constexpr int PART = 16 * ROW;                // bytes of 16 tokens of K or V
    // 16-token parts of a tile: two, so that a warp has two independent chains of products
    // and half the work around them (8 heads with probes: 134 -> 121 us); one of 256-byte
    // rows, where two stages of two would leave one CTA per SM
    static constexpr int SUBS = Q8 || D == 64 ? 2 : 1;
    static constexpr int TILE_TOKENS = 16 * SUBS;
    static constexpr int HALF = SUBS * PART;             // bytes of a K or V tile
    static constexpr int TILE_BYTES = 2 * HALF;
    static constexpr int QUAD = WARPS * TILE_TOKENS;     // tokens of one tile per warp: the schedule's step
    static constexpr int STAGES = TILE_BYTES <= 4096 ? 3 : 2;            // tiles of a warp's ring
    // CTAs per SM that registers (128, 168 and 255 a thread) and rings leave room for.
    // Measured at d = 128, 16-token tiles (per-head cache above): 4 CTAs of 2 stages 176 us,
    // 3 of 4 181, 4 of 3 191; 32-token tiles, 3 of 2: 176.  Two n-tiles: 3 CTAs would spill
    // at d = 128 (125 against 120 us) and do not at d = 64 (29.0 against 29.5).
    static constexpr int CTAS = NT == 2 && D == 128 ? 2 : (NT == 1 && Q8 && D == 64 ? 4 : 3);
    static constexpr int RING_BYTES = WARPS * STAGES * TILE_BYTES;
    static constexpr int BAR_OFF = RING_BYTES > MERGE_BYTES ? RING_BYTES : MERGE_BYTES;
    static constexpr int SMEM = BAR_OFF + 8 * WARPS * STAGES + 1024;     // and what aligning the base to 1024 takes
};

// Floats of a cut item's part per head: O[D] (and M[D]).
template <int D, bool RHO> constexpr int part_stride() { return (RHO ? 2 : 1) * D; }

// Scratch of a call, in the order of DecodeCacheScratch.
struct Scratch {
    float *parts;       // [slot][HEADS][O, M]
    float4 *hdr;        // [slot][HEADS] (m, l, abar) of the cut items' parts
    int2 *cut;          // [CTA] (item, parts) of the item it starts but does not finish, or (-1, 0)
    int2 *item;         // [item] (first CTA, parts)
    float *lse2;        // [B, Hq] log2 of an uncut item's sum, with weights
    float *zs;          // [item][Tcap][HEADS] scores (log2), with weights
};

template <int D, bool Q8, bool RHO, int NT, typename Tout>
__global__ void __launch_bounds__(WARPS * 32, Shape<D, Q8, RHO, NT>::CTAS) k_decode_cache(
    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
    const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ rho, const signed char *__restrict__ kexp,
    const signed char *__restrict__ vexp, const int *__restrict__ seqlens, Tout *__restrict__ y, float *__restrict__ lse,
    int B, int Hq, int htiles, Split split, PagedKV pg, Scratch ws, DeviceCtl ctl) {
    using S = Shape<D, Q8, RHO, NT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023) & 1023);
    float *merge = reinterpret_cast<float *>(smem);
    __shared__ int abort_flag;
    __shared__ long long wsum[WARPS], sh_before;
    __shared__ int sh_b;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t full = smem_u32(smem + S::BAR_OFF) + 8 * S::STAGES * warp;     // this warp's barriers, one per stage
    const int r = lane / 4, t4 = lane % 4;
    const float scale_log2 = LOG2E / sqrtf((float)D);
    const int ps = 1 << pg.pshift, pmask = ps - 1;
    const int Tcap = pg.max_pages << pg.pshift;
    const int per_seq = pg.Hkv * htiles;     // items of a sequence
    auto len_of = [&](int i) { return min(max(seqlens[i], 0), Tcap); };

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    // whole items, by the CTA or by each of its warps alone: tiles first_w, first_w + step_w, ..
    const bool whole = split != Split::RANGES, solo = split == Split::WARPS;
    const int first_w = solo ? 0 : warp, step_w = solo ? 1 : WARPS;
    if (threadIdx.x == 0) abort_flag = 0;
    if (lane == 0)
        for (int i = 0; i < S::STAGES; ++i) mbar_init(full + 8 * i, 1);
    fence_mbar_init();
    __syncthreads();                         // the last of the CTA in solo mode
    // ---- this CTA's range of quads: from quad `q0` of item `it` of sequence `b`, `left` quads ----
    int b, it, q0 = 0, cta = 0, nctas = 1;
    long long left, pos = 0, total = 1;
    if (whole) {
        const int x = solo ? blockIdx.x * WARPS + warp : blockIdx.x;
        b = x / per_seq;                     // B for a warp without an item
        it = x % per_seq;
        left = b < B ? quads_of(len_of(b), S::QUAD) : 0;
    } else {
        // prefix sums of the sequences' quads: a run of sequences per thread, then over the threads
        const int run = (B + WARPS * 32 - 1) / (WARPS * 32);
        const int b0 = min((int)threadIdx.x * run, B), b1 = min(b0 + run, B);
        long long own = 0;
#pragma unroll 8
        for (int i = b0; i < b1; ++i) own += quads_of(len_of(i), S::QUAD);
        long long incl = own;
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
            const long long o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        long long all = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w == warp) incl += all;
            all += wsum[w];
        }
        total = all * per_seq;
        cta = blockIdx.x;
        nctas = sched_ctas(total, gridDim.x);
        if (threadIdx.x == 0) ws.cut[cta] = make_int2(-1, 0);
        if (cta >= nctas) {
            left = 0;
        } else {
            pos = sched_start(cta, total, nctas);
            left = sched_start(cta + 1, total, nctas) - pos;
            long long before = incl - own;
            if (before * per_seq <= pos && pos < incl * per_seq) {
                int i = b0;
                for (int n; (before + (n = quads_of(len_of(i), S::QUAD))) * per_seq <= pos; ++i) before += n;
                sh_b = i;
                sh_before = before;
            }
            __syncthreads();
            b = sh_b;
            const long long rem = pos - sh_before * per_seq;
            const int n = quads_of(len_of(b), S::QUAD);
            it = (int)sched_div(rem, n);
            q0 = (int)(rem - (long long)it * n);
        }
    }
    // sequences without a token: nothing else writes their rows
    for (int e = whole ? b : (int)blockIdx.x; e < B; e += whole ? B : (int)gridDim.x) {
        if (len_of(e) > 0 || (whole && it != 0)) continue;
        for (int i = first_w * 32 + lane; i < Hq * D; i += step_w * 32) store_y<Tout>(y + (size_t)e * Hq * D + i, 0.f);
        if (lse != nullptr)
            for (int i = first_w * 32 + lane; i < Hq; i += step_w * 32) lse[(size_t)e * Hq + i] = -INFINITY;
    }
    if (left == 0) return;

    const WaitCtl wait{ctl.err, &abort_flag, ctl.wait_ns};
    int stage = 0;               // stage of this warp's next tile
    uint32_t phases = 0;         // parity each stage's barrier completes next

    while (true) {
        const int L = len_of(b), nq = quads_of(L, S::QUAD);
        const int q1 = (int)min((long long)nq, q0 + left);
        const int kvh = it / htiles, ht = it % htiles;
        const int g0 = ht * S::HEADS;
        const int nh = min(S::HEADS, pg.group - g0);
        const long h0 = (long)b * Hq + (long)kvh * pg.group + g0;
        const long item = (long)b * per_seq + it;
        const int t0 = q0 * S::QUAD;
        const int t1 = min(L, q1 * S::QUAD);
        const int ntiles = (t1 - t0 + S::TILE_TOKENS - 1) / S::TILE_TOKENS;
        const bool uncut = q0 == 0 && q1 == nq;

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
        // O is held at 2^(mref + oexp), M at that over mratio, both times 2^WSHIFT (e4m3)
        int oexp[S::HPT];
        float mratio[S::HPT];
#pragma unroll
        for (int i = 0; i < S::HPT; ++i) {
            oexp[i] = -400;       // below any that a tile sets
            mratio[i] = 1.f;
        }

        // This warp's tiles are first_w + step_w j.  Lane l holds the page of its 16-token part
        // 32 n + l (a part's rows share one page: it starts on a multiple of 16 and pages
        // hold at least 16) and its two exponents, loaded 32 parts at a time.
        const int mine = ntiles > first_w ? (ntiles - first_w + step_w - 1) / step_w : 0;
        auto token_of = [&](int part) {
            return t0 + (first_w + step_w * (part / S::SUBS)) * S::TILE_TOKENS + (part % S::SUBS) * 16;
        };
        // (read up to the table's end: the entries past t1 are not followed, and their load does not wait
        // for the length)
        auto page_of = [&](int part) -> int {
            const int t = token_of(part);
            return t < Tcap ? pg.table[(size_t)b * pg.max_pages + (t >> pg.pshift)] : 0;
        };
        // exponents of K (low byte) and V (next byte), and BAD for a page id out of range
        auto info_of = [&](int part, int id) -> int {
            const int t = token_of(part);
            if (t >= t1) return NO_EXPONENTS;
            if ((unsigned)id >= (unsigned)pg.num_pages) {
                atomicExch(ctl.err, PARALLAX_ERR_DEVICE_INDEX);
                return BAD | NO_EXPONENTS;
            }
            if constexpr (!Q8) return 0;
            const size_t at = ((size_t)id * pg.Hkv + kvh) * (ps / KV_BLOCK) + (t & pmask) / KV_BLOCK;
            return (kexp[at] & 0xff) | (vexp[at] & 0xff) << 8;
        };
        int ids = page_of(lane), ids_next = 0;
        // the vectors, column n = r of n-tile nt, as they are: loaded before anything waits for the pages
        uint2 qw[NT][S::KSTEPS];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int head = RHO ? nt * 4 + r / 2 : nt * 8 + r;
            const bool live = head < nh;
            const __nv_bfloat16 *src = (RHO && (r & 1) ? rho : q) + (h0 + (live ? head : 0)) * D;
#pragma unroll
            for (int s = 0; s < S::KSTEPS; ++s) {
                const int d0 = Q8 ? 64 * (s / 4) + 16 * t4 + 4 * (s % 4) : 32 * (s / 2) + 8 * t4 + 4 * (s % 2);
                qw[nt][s] = live ? *reinterpret_cast<const uint2 *>(src + d0) : make_uint2(0u, 0u);
            }
        }
        int info = info_of(lane, ids), info_next = 0;

        uint8_t *ring = smem + warp * S::STAGES * S::TILE_BYTES;
        // Loads tile j into stage st; lane l holds the page of part 32 n + l in `pages`.
        // Parts past the end and those of a bad page are not loaded.
        auto issue = [&](int j, int st, int pages) {
            int id[S::SUBS], bytes = 0;
            bool ok[S::SUBS];
#pragma unroll
            for (int u = 0; u < S::SUBS; ++u) {
                id[u] = __shfl_sync(0xffffffffu, pages, (S::SUBS * j + u) & 31);
                ok[u] = (unsigned)id[u] < (unsigned)pg.num_pages && token_of(S::SUBS * j + u) < t1;
                bytes += ok[u] ? 2 * S::PART : 0;
            }
            __syncwarp();                        // every lane has read what the stage held
            if (lane == 0) {
                const bool skip = (ctl.debug_flags & DEBUG_DECODE_SKIP_FIRST_TILE) && j == 0;
                mbar_arrive_expect_tx(full + 8 * st, bytes);
#pragma unroll
                for (int u = 0; u < S::SUBS; ++u) {
                    if (!ok[u] || skip) continue;
                    const uint32_t dst = smem_u32(ring + st * S::TILE_BYTES + u * S::PART);
                    const int row = token_of(S::SUBS * j + u) & pmask, slab = id[u] * pg.Hkv + kvh;
#pragma unroll
                    for (int x = 0; x < S::BOXES; ++x) {
                        tma_load_3d(dst + x * 16 * S::RB, &tmk, full + 8 * st, x * (S::RB / S::EL), row, slab);
                        tma_load_3d(dst + S::HALF + x * 16 * S::RB, &tmv, full + 8 * st, x * (S::RB / S::EL), row, slab);
                    }
                }
            }
        };
#pragma unroll
        for (int j = 0; j < S::STAGES - 1; ++j)
            if (j < mine) issue(j, (stage + j) % S::STAGES, ids);
        // ---- the vectors (the first tiles are on their way): column n = r of n-tile nt; 4 elements per MMA step ----
        uint32_t qf[NT][S::KSTEPS][2];
        float zfac[S::HPT], afac[S::HPT] = {};    // of the heads whose state this thread holds
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint2 *w = qw[nt];
            uint32_t big = 0;
#pragma unroll
            for (int s = 0; s < S::KSTEPS; ++s) {
                big = max(big, max(max(w[s].x & 0x7fffu, w[s].x >> 16 & 0x7fffu), max(w[s].y & 0x7fffu, w[s].y >> 16 & 0x7fffu)));
            }
            float inv = 1.f;
            if constexpr (Q8) {
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                // bring the largest element to [2^7, 2^8), or 2^120 closer: subnormal ones are exact there
                const int up = min(max(134 - (int)(big >> 7), -120), 120);
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

        // where this thread's tokens and chunks lie in a tile
        const int tok0 = row_of<S::RB>(r), tok1 = tok0 + 8;
        const int koff = chunk_at<S::RB>(tok0, t4);
        const int va = row_of<S::RB>(2 * t4), vb = row_of<S::RB>(2 * t4 + 1);
        const int vc = S::VB < 16 ? r / 2 : r, vsub = S::VB < 16 ? 8 * (r & 1) : 0;
        const int voff[2] = {S::HALF + chunk_at<S::RB>(va, vc) + vsub, S::HALF + chunk_at<S::RB>(vb, vc) + vsub};
        bool gave_up = false;
        for (int j = 0; j < mine; ++j) {
            // ---- pages and exponents of the 32 parts after these, in good time ----
            constexpr int PER32 = 32 / S::SUBS;
            if (j % PER32 == 0)
                ids_next = page_of(S::SUBS * (j + PER32) + lane);
            else if (j % PER32 == PER32 / 2)
                info_next = info_of(S::SUBS * (j + PER32 / 2) + lane, ids_next);
            const int jn = j + S::STAGES - 1;
            // every lane has read the tile before this one: its stage takes tile jn
            if (jn < mine) issue(jn, stage == 0 ? S::STAGES - 1 : stage - 1, j % PER32 + S::STAGES - 1 < PER32 ? ids : ids_next);
            int ke[S::SUBS], ve[S::SUBS];
            bool bad = false;
#pragma unroll
            for (int u = 0; u < S::SUBS; ++u) {
                const int now = __shfl_sync(0xffffffffu, info, (S::SUBS * j + u) & 31);
                ke[u] = (int)(signed char)now;
                ve[u] = (int)(signed char)(now >> 8);
                bad |= (now & BAD) != 0;
            }
            const int parts_info = info;
            if (j % PER32 == PER32 - 1) {
                ids = ids_next;
                info = info_next;
            }
            const bool landed = mbar_wait(full + 8 * stage, (phases >> stage) & 1u, wait);
            if (!__all_sync(0xffffffffu, landed)) {
                gave_up = true;
                // give up: let this warp's copies land (bounded) before the CTA's memory goes
                for (int i = j; i < min(jn + 1, mine); ++i) {
                    const int st = (stage + i - j) % S::STAGES;
                    mbar_wait_drain(full + 8 * st, (phases >> st) & 1u, 2000000ull);
                }
                break;
            }
            phases ^= 1u << stage;
            uint8_t *dk = ring + stage * S::TILE_BYTES;
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
            const int tile = token_of(S::SUBS * j);
            const int nvalid = t1 - tile;                   // tokens of the tile
            const bool ragged = nvalid < S::TILE_TOKENS;
            if (ragged || bad) {
                // rows past the sequence hold whatever the page does, those of a bad page or a part
                // past the end what the stage held: zeros, as a weight of 0 times NaN is no 0
#pragma unroll
                for (int u = 0; u < S::SUBS; ++u) {
                    const bool out = (__shfl_sync(0xffffffffu, parts_info, (S::SUBS * j + u) & 31) & BAD) != 0;
                    for (int i = lane; i < 2 * S::PART / 16; i += 32) {
                        const int kv = i / (S::PART / 16), at = i % (S::PART / 16) * 16;      // K or V, byte of the part
                        if (out || 16 * u + at / S::RB % 16 >= nvalid)
                            *reinterpret_cast<uint4 *>(dk + kv * S::HALF + u * S::PART + at) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async();               // before a later load into this stage
                __syncwarp();
            }

            // ---- scores: two chains of products, one per part or by turns ----
            constexpr int CHAINS = S::SUBS == 1 ? 2 : 1;
            float sc[S::SUBS][NT][4], sc2[S::SUBS][NT][4];
#pragma unroll
            for (int u = 0; u < S::SUBS; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[u][nt][e] = sc2[u][nt][e] = 0.f;
#pragma unroll
            for (int c = 0; c < S::KC; ++c) {
                alignas(16) uint32_t w0[S::SUBS][4], w1[S::SUBS][4];
#pragma unroll
                for (int u = 0; u < S::SUBS; ++u) {
                    const uint8_t *src = dk + u * S::PART + (c / 2) * 16 * S::RB + (koff ^ ((c & 1) << 6));
                    *reinterpret_cast<uint4 *>(w0[u]) = *reinterpret_cast<const uint4 *>(src);
                    *reinterpret_cast<uint4 *>(w1[u]) = *reinterpret_cast<const uint4 *>(src + 8 * S::RB);
                }
#pragma unroll
                for (int i = 0; i < (Q8 ? 4 : 2); ++i)
#pragma unroll
                    for (int u = 0; u < S::SUBS; ++u) {
                        const int st = c * (Q8 ? 4 : 2) + i;
                        uint32_t a0, a1, a2, a3;
                        if constexpr (Q8) {
                            e4m3x4_to_f16x2(w0[u][i], a0, a2);
                            e4m3x4_to_f16x2(w1[u][i], a1, a3);
                        } else {
                            a0 = w0[u][2 * i];
                            a2 = w0[u][2 * i + 1];
                            a1 = w1[u][2 * i];
                            a3 = w1[u][2 * i + 1];
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<Q8>(CHAINS == 2 && st % 2 ? sc2[u][nt] : sc[u][nt], a0, a1, a2, a3, qf[nt][st][0],
                                         qf[nt][st][1]);
                    }
            }
            if constexpr (CHAINS == 2) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[0][nt][e] += sc2[0][nt][e];
            }

            // ---- weights ----
            constexpr int ROWS = 2 * S::SUBS;     // a thread's tokens: row x is 16 (x / 2) + (x odd ? tok1 : tok0)
            auto tok = [&](int x) { return 16 * (x >> 1) + ((x & 1) ? tok1 : tok0); };
            float f[S::SUBS][S::HPT], fa[S::SUBS][S::HPT];       // z = sc * f, a = sc * fa
#pragma unroll
            for (int u = 0; u < S::SUBS; ++u) {
                const float kscale = Q8 ? exp2_whole(ke[u]) : 1.f;
#pragma unroll
                for (int h = 0; h < S::HPT; ++h) {
                    f[u][h] = Q8 ? fminf(zfac[h] * kscale, 3e38f) : zfac[h];         // finite: a score of 0 stays 0
                    fa[u][h] = Q8 ? fminf(afac[h] * kscale, 3e38f) : afac[h];
                }
            }
            auto score = [&](int h, int x) { return sc[x >> 1][RHO ? h : h / 2][2 * (x & 1) + (RHO ? 0 : h % 2)]; };
            auto masked = [&](int x) { return ragged && tok(x) >= nvalid; };
            auto weight = [&](int h, int x) {
                const float dz = fmaf(score(h, x), f[x >> 1][h], -mref[h]);
                return fex2(masked(x) ? -INFINITY : dz);
            };
            auto probe = [&](int h, int x) { return sc[x >> 1][h][2 * (x & 1) + 1] * fa[x >> 1][h]; };
            // weights: p against mref, and those of O and M as they are held (masked tokens have p = 0
            // and, their K rows being zero, a = 0); whether one has outgrown its reference (NaN does not)
            float p[S::HPT][ROWS], wo[S::HPT][ROWS], wm[S::HPT][ROWS];
            auto weigh = [&] {
                bool up = false;
#pragma unroll
                for (int h = 0; h < S::HPT; ++h) {
                    float top = 0.f, topw = 0.f;
#pragma unroll
                    for (int x = 0; x < ROWS; ++x) {
                        p[h][x] = weight(h, x);
                        top = fmaxf(top, p[h][x]);
                        wo[h][x] = Q8 ? p[h][x] * exp2_whole(min(ve[x >> 1] - oexp[h] + WSHIFT, 126)) : p[h][x];
                        topw = fmaxf(topw, wo[h][x]);
                        if constexpr (RHO) {
                            wm[h][x] = wo[h][x] * probe(h, x);
                            if constexpr (Q8) wm[h][x] *= mratio[h];
                            topw = fmaxf(topw, fabsf(wm[h][x]));
                        }
                    }
                    up |= top > HEADROOM;
                    if constexpr (Q8) up |= topw > HEADROOM * (1 << WSHIFT);
                }
                return up;
            };
            if (ws.zs != nullptr) {
                float *dst = ws.zs + ((size_t)item * Tcap + tile) * S::HEADS;
#pragma unroll
                for (int h = 0; h < S::HPT; ++h) {
                    const int head = RHO ? 4 * h + t4 : 8 * (h / 2) + 2 * t4 + h % 2;
#pragma unroll
                    for (int x = 0; x < ROWS; ++x)
                        if (tok(x) < nvalid) dst[tok(x) * S::HEADS + head] = score(h, x) * f[x >> 1][h];
                }
            }
            // (a warp's first tile always sets the references: a short call does not wait for the
            // instructions of a first try, 12.5 against 14.3 us for one tile per warp)
            if (j == 0 || __any_sync(0xffffffffu, weigh())) {
#pragma unroll
                for (int h = 0; h < S::HPT; ++h) {
                    const int nt = RHO ? h : h / 2, e = RHO ? 0 : h % 2;
                    float top = -INFINITY;
#pragma unroll
                    for (int x = 0; x < ROWS; ++x) top = fmaxf(top, masked(x) ? -INFINITY : score(h, x) * f[x >> 1][h]);
#pragma unroll
                    for (int off = 4; off < 32; off *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    const float mnew = fmaxf(mref[h], top), down = mref[h] - mnew;
                    const float alpha = fex2(down);
                    mref[h] = mnew;
                    lsum[h] *= alpha;
                    asum[h] *= alpha;
                    float bo = alpha, bm = alpha;                  // what O and M held so far becomes
                    if constexpr (Q8) {
                        // The whole exponents above the tile's largest p 2^ve and p |a| 2^ve: both maxima at
                        // once, in the upper halves of their floats (one that underflows is below any that counts)
                        float o = 0.f, m = 0.f;
#pragma unroll
                        for (int x = 0; x < ROWS; ++x) {
                            const float w = weight(h, x) * exp2_whole(ve[x >> 1]);
                            o = fmaxf(o, w);
                            if constexpr (RHO) m = fmaxf(m, w * fabsf(probe(h, x)));
                        }
                        uint32_t both = __byte_perm(__float_as_uint(o), __float_as_uint(m), 0x7632);
#pragma unroll
                        for (int off = 4; off < 32; off *= 2) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, off));
                        const int fell = __float2int_rd(fmaxf(down, -1e3f));     // (down: a reference never creeps up)
                        const int eo = max((int)(both >> 7 & 255) - 126, oexp[h] + fell);
                        bo = fex2(down + (float)(oexp[h] - eo));
                        if constexpr (RHO) {
                            const int held = oexp[h] - whole_log2(mratio[h]);
                            const int em = min(max(max((int)(both >> 23) - 126, held + fell), eo - 30), eo + 126);
                            bm = fex2(down + (float)(held - em));
                            mratio[h] = exp2_whole(eo - em);
                        }
                        oexp[h] = eo;
                    }
#pragma unroll
                    for (int i = 0; i < S::JS; ++i) {
                        if constexpr (RHO) {
                            oacc[nt][i][0] *= bo;
                            oacc[nt][i][1] *= bm;
                            oacc[nt][i][2] *= bo;
                            oacc[nt][i][3] *= bm;
                        } else {
                            oacc[nt][i][e] *= bo;
                            oacc[nt][i][2 + e] *= bo;
                        }
                    }
                }
                weigh();
            }
            uint32_t bh[NT][ROWS], bl[NT][ROWS];    // weights as the value product's operand: hi, lo parts
#pragma unroll
            for (int x = 0; x < ROWS; ++x) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t hi, lo;
                    if constexpr (RHO) {
                        lsum[nt] += p[nt][x];
                        asum[nt] = fmaf(p[nt][x], probe(nt, x), asum[nt]);
                        split_pair<Q8>(wo[nt][x], wm[nt][x], hi, lo);
                    } else {
                        lsum[2 * nt] += p[2 * nt][x];
                        lsum[2 * nt + 1] += p[2 * nt + 1][x];
                        split_pair<Q8>(wo[2 * nt][x], wo[2 * nt + 1][x], hi, lo);
                    }
                    bh[nt][x] = movmatrix(hi);
                    bl[nt][x] = movmatrix(lo);
                }
            }
            // ---- O += P V, M += (P o A) V ----
#pragma unroll
            for (int cu = 0; cu < (S::VB + 15) / 16 * S::SUBS; ++cu) {
                const int c = cu / S::SUBS, u = cu % S::SUBS;
                alignas(16) uint32_t v[4][4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {       // tokens of the weights' columns 2 t4, 2 t4 + 1, + 8, + 9
                    const uint8_t *src = dk + u * S::PART + c * 16 * S::RB + voff[x & 1] + 8 * (x >> 1) * S::RB;
                    if constexpr (S::VB < 16)
                        *reinterpret_cast<uint2 *>(v[x]) = *reinterpret_cast<const uint2 *>(src);
                    else
                        *reinterpret_cast<uint4 *>(v[x]) = *reinterpret_cast<const uint4 *>(src);
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
                                             part ? bl[nt][2 * u] : bh[nt][2 * u], part ? bl[nt][2 * u + 1] : bh[nt][2 * u + 1]);
                }
            }
        }
        // O and M of head h as they are, for what the accumulators hold
        auto of_o = [&](float v, int h) { return Q8 ? scaled(v, oexp[h] - WSHIFT) : v; };
        auto of_m = [&](float v, int h) { return Q8 ? scaled(v, oexp[h] - whole_log2(mratio[h]) - WSHIFT) : v; };
        if (solo) {
            // the item is this warp's alone: the thread that holds a head's O[d] also holds its M[d]
            if (gave_up) return;
#pragma unroll
            for (int h = 0; h < S::HPT; ++h) {
                const int head = RHO ? 4 * h + t4 : 8 * (h / 2) + 2 * t4 + h % 2, nt = RHO ? h : h / 2;
                float l = lsum[h], ab = asum[h];
#pragma unroll
                for (int off = 4; off < 32; off *= 2) {
                    l += __shfl_xor_sync(0xffffffffu, l, off);
                    ab += __shfl_xor_sync(0xffffffffu, ab, off);
                }
                if (head >= nh) continue;
                const float inv = 1.f / l, c = ab * inv;
                Tout *yr = y + (h0 + head) * D;
#pragma unroll
                for (int j = 0; j < S::JS; ++j) {
                    const int d = Q8 || S::VB == 16 ? (S::VB / S::EL) * r + 2 * j : 64 * (j / 4) + 8 * r + 2 * (j % 4);
                    if constexpr (RHO) {
                        const float o0 = of_o(oacc[nt][j][0] * inv, h), o1 = of_o(oacc[nt][j][2] * inv, h);
                        store_y2(yr + d, o0 - (of_m(oacc[nt][j][1] * inv, h) - o0 * c),
                                 o1 - (of_m(oacc[nt][j][3] * inv, h) - o1 * c));
                    } else {
                        store_y2(yr + d, of_o(oacc[nt][j][h % 2] * inv, h), of_o(oacc[nt][j][2 + h % 2] * inv, h));
                    }
                }
                if (r == 0) {
                    const float l2 = mref[h] + log2f(l);
                    if (lse != nullptr) lse[h0 + head] = l2 * LN2;
                    if (ws.lse2 != nullptr) ws.lse2[h0 + head] = l2;
                    if (ws.item != nullptr && h == 0 && t4 == 0) ws.item[item] = make_int2(0, 1);
                }
            }
            return;
        }
        __syncthreads();   // every warp is done with its ring: reuse it for the merge
        if (abort_flag) return;

        // ---- merge the warps' states per head ----
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
                    row[4 + d] = of_o(oacc[nt][j][0], h);
                    row[4 + d + 1] = of_o(oacc[nt][j][2], h);
                    row[4 + D + d] = of_m(oacc[nt][j][1], h);
                    row[4 + D + d + 1] = of_m(oacc[nt][j][3], h);
                } else {
                    row[4 + d] = of_o(oacc[nt][j][h % 2], h);
                    row[4 + d + 1] = of_o(oacc[nt][j][2 + h % 2], h);
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
            if (uncut) {
                const float inv = 1.0f / l;
                float out = o * inv;
                if constexpr (RHO) out -= m * inv - out * (ab * inv);
                store_y<Tout>(y + bh * D + e, out);
                if (e == 0) {
                    const float l2 = mu + log2f(l);
                    if (lse != nullptr) lse[bh] = l2 * LN2;
                    if (ws.lse2 != nullptr) ws.lse2[bh] = l2;
                }
            } else {
                const int slot = sched_slot(cta, q0 == 0) * S::HEADS + hh;
                float *P = ws.parts + (size_t)slot * part_stride<D, RHO>();
                P[e] = o;
                if constexpr (RHO) P[D + e] = m;
                if (e == 0) ws.hdr[slot] = make_float4(mu, l, ab, 0.f);
            }
        }
        if (q0 == 0 && threadIdx.x == 0) {
            const int parts = uncut ? 1 : sched_owner(pos + nq - 1, total, nctas) - cta + 1;
            if (!uncut) ws.cut[cta] = make_int2((int)item, parts);
            if (ws.item != nullptr) ws.item[item] = make_int2(cta, parts);
        }
        left -= q1 - q0;
        if (left == 0) break;
        pos += q1 - q0;
        q0 = 0;
        if (++it == per_seq) {
            it = 0;
            do ++b;
            while (len_of(b) == 0);
        }
        fence_proxy_async();   // the next item's copies write where these stores and loads went
        __syncthreads();
    }
}

// n / d for n < 2^31 by a multiplication (d >= 1): m = ceil(2^(31 + s) / d) with 2^s >= d
// (T. Granlund, P. L. Montgomery, Division by Invariant Integers using Multiplication, 1994).
struct Divisor {
    unsigned d, m, s;
    explicit Divisor(int n) : d(n > 0 ? (unsigned)n : 1u), s(0) {
        while ((1ull << s) < d) ++s;
        m = (unsigned)(((1ull << (31 + s)) + d - 1) / d);
    }
    __device__ __forceinline__ unsigned of(unsigned n) const { return (unsigned)(((unsigned long long)n * m) >> (31 + s)); }
};

constexpr int FIN_THREADS = 256;
constexpr int ACC_TOKENS = 1024;

// One launch after the decode (a programmatic dependent: its blocks are there when
// the decode's CTAs leave).  The first blocks merge cut items and write y and lse:
// one per CTA of the decode (the item that CTA starts but does not finish) with all
// its heads, or, when items are few and have many parts (hpb = 1), one per item
// and head; the others add the weights s = 2^(z - lse2) of ACC_TOKENS tokens of
// one (b, kvh) to the accumulator, summed over the KV head's query heads in head
// order (each token by one thread: the result does not depend on the schedule).
template <int D, bool RHO, int HEADS, typename Tout>
__global__ void __launch_bounds__(FIN_THREADS, 4) k_decode_finish(
    Scratch ws, const int *__restrict__ seqlens, Tout *__restrict__ y, float *__restrict__ lse, float *__restrict__ wacc,
    int Hq, int Hkv, int htiles, int Tcap, int ctas, int hpb, int combine_blocks, Divisor by_chunks, Divisor by_heads) {
    constexpr int COLS = (RHO ? 2 : 1) * D / 4;               // float4 columns of a part
    constexpr int GROUPS = FIN_THREADS / COLS;                // thread groups of one column each
    __shared__ float4 red[GROUPS][COLS];
    __shared__ float4 redl[GROUPS];
    __shared__ __align__(16) float slse[HEADS];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int group = Hq / Hkv;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x < combine_blocks) {
        const int at = blockIdx.x / (HEADS / hpb), hfirst = blockIdx.x % (HEADS / hpb) * hpb;
        const int per_seq = Hkv * htiles;
        int item, c0, nv;                                     // the cut item, its first CTA and its parts
        if (hpb == 1) {
            const int2 info = ws.item[at];
            item = at;
            c0 = info.x;
            nv = info.y;
            // not written: an empty sequence, or a decode that gave up on a wait
            if (seqlens[at / per_seq] <= 0 || c0 < 0 || c0 >= ctas || nv < 2 || nv > ctas - c0) return;
        } else {
            const int2 cut = ws.cut[at];
            item = cut.x;
            c0 = at;
            nv = cut.y;
            if (item < 0) return;
        }
        const int b = item / per_seq, it = item % per_seq;
        const int g0 = (it % htiles) * HEADS;
        const long bh0 = (long)b * Hq + (long)(it / htiles) * group + g0;
        const int col = tid % COLS, grp = tid / COLS;
        // `by` groups share a head's parts: all of them when a block has one head, else one each
        const int by = hpb == 1 ? GROUPS : 1, heads = GROUPS / by;
        for (int h1 = hfirst; h1 < hfirst + hpb; h1 += heads) {
            const int hh = h1 + grp / by;
            const bool live = hh < hfirst + hpb && g0 + hh < group;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f, ab = 0.f, mu = MNONE;
            if (live) {
                // header and part of four parts at a time, against the group's own maximum so far
                const float4 *P = reinterpret_cast<const float4 *>(ws.parts) + col;
                for (int s0 = grp % by; s0 < nv; s0 += 4 * by) {
                    float4 h[4], p[4];
                    float top = mu;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int s = s0 + i * by;
                        const int slot = sched_part(c0, s < nv ? s : s0) * HEADS + hh;
                        h[i] = ws.hdr[slot];
                        p[i] = P[(size_t)slot * COLS];
                        if (s >= nv) h[i].x = -INFINITY;       // weighs 0
                        top = fmaxf(top, h[i].x);
                    }
                    const float down = fex2(mu - top);
                    mu = top;
                    l *= down;
                    ab *= down;
                    acc = make_float4(acc.x * down, acc.y * down, acc.z * down, acc.w * down);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w = fex2(h[i].x - mu);
                        l = fmaf(w, h[i].y, l);
                        ab = fmaf(w, h[i].z, ab);
                        acc.x = fmaf(w, p[i].x, acc.x);
                        acc.y = fmaf(w, p[i].y, acc.y);
                        acc.z = fmaf(w, p[i].z, acc.z);
                        acc.w = fmaf(w, p[i].w, acc.w);
                    }
                }
            }
            __syncthreads();
            red[grp][col] = acc;
            if (col == 0) redl[grp] = make_float4(l, ab, mu, 0.f);
            __syncthreads();
            if (live) {
                const int first = grp / by * by;              // the groups of this head
                for (int i = 0; i < by; ++i) mu = fmaxf(mu, redl[first + i].z);
                float w[GROUPS];
                l = ab = 0.f;
#pragma unroll
                for (int i = 0; i < GROUPS; ++i) {
                    if (i >= by) break;
                    w[i] = fex2(redl[first + i].z - mu);
                    l = fmaf(w[i], redl[first + i].x, l);
                    ab = fmaf(w[i], redl[first + i].y, ab);
                }
                const float inv = 1.f / l;
                const float *R = reinterpret_cast<const float *>(red[first]);
                for (int e = tid - first * COLS; e < D; e += by * COLS) {
                    float o = 0.f, m = 0.f;
#pragma unroll
                    for (int i = 0; i < GROUPS; ++i) {
                        if (i >= by) break;
                        o = fmaf(w[i], R[i * COLS * 4 + e], o);
                        if constexpr (RHO) m = fmaf(w[i], R[i * COLS * 4 + D + e], m);
                    }
                    float out = o * inv;
                    if constexpr (RHO) out -= m * inv - out * (ab * inv);
                    store_y<Tout>(y + (bh0 + hh) * D + e, out);
                    if (e == 0 && lse != nullptr) lse[bh0 + hh] = (mu + log2f(l)) * LN2;
                }
            }
        }
        return;
    }
    // ---- accumulate: every load whose address is known is issued first ----
    const unsigned rest = blockIdx.x - combine_blocks;
    const unsigned bk = by_chunks.of(rest);                    // b * Hkv + kvh
    const int t0 = (int)(rest - bk * by_chunks.d) * ACC_TOKENS;
    const int b = (int)by_heads.of(bk), kvh = (int)(bk - (unsigned)b * Hkv);
    constexpr int PER = ACC_TOKENS / FIN_THREADS;
    const int L = min(max(seqlens[b], 0), Tcap);
    const size_t row = (size_t)bk * Tcap + t0 + tid;
    float *W = wacc + row;
    float sum[PER], add[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) add[k] = 0.f;
    // `full`: no token of the chunk lies past the table (their scratch and weights may be
    // read, also past the sequence's end, but only tokens before it are written)
    auto run = [&](auto full_, auto htiles_) {
        constexpr bool FULL = decltype(full_)::value;
        const int nht = decltype(htiles_)::value ? 1 : htiles;
        const int room = Tcap - t0 - tid;
#pragma unroll
        for (int k = 0; k < PER; ++k) sum[k] = FULL || k * FIN_THREADS < room ? W[k * FIN_THREADS] : 0.f;
        for (int ht = 0; ht < nht; ++ht) {
            const int nh = min(HEADS, group - ht * HEADS);
            const int item = (int)bk * nht + ht;
            const long h0 = (long)b * Hq + (long)kvh * group + ht * HEADS;
            const float4 *Z = reinterpret_cast<const float4 *>(ws.zs) +
                              ((size_t)item * Tcap + t0 + tid) * (HEADS / 4);
            float4 z[PER][HEADS / 4];
#pragma unroll
            for (int k = 0; k < PER; ++k)
#pragma unroll
                for (int c = 0; c < HEADS / 4; ++c)
                    z[k][c] = FULL || k * FIN_THREADS < room ? Z[k * FIN_THREADS * (HEADS / 4) + c]
                                                             : make_float4(0.f, 0.f, 0.f, 0.f);
            int2 info = ws.item[item];
            const float l2 = lane < nh ? ws.lse2[h0 + lane] : 0.f;       // of an uncut item
            if (t0 >= L) return;
            // a decode that gave up on a wait has not written it: whatever is read stays in bounds
            if (info.x < 0 || info.x >= ctas || info.y < 1 || info.y > ctas - info.x) info = make_int2(0, 1);
            if (ht > 0) __syncthreads();
            if (info.y == 1) {
                if (tid < nh) slse[tid] = l2;
            } else {
                for (int h = warp; h < nh; h += FIN_THREADS / 32) {
                    float top = MNONE, l = 0.f;
                    for (int s = lane; s < info.y; s += 32) {
                        const float4 p = ws.hdr[sched_part(info.x, s) * HEADS + h];
                        const float m = fmaxf(top, p.x);
                        l = l * fex2(top - m) + fex2(p.x - m) * p.y;
                        top = m;
                    }
                    float mu = top;
#pragma unroll
                    for (int off = 16; off > 0; off /= 2) mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, off));
                    l *= fex2(top - mu);
#pragma unroll
                    for (int off = 16; off > 0; off /= 2) l += __shfl_xor_sync(0xffffffffu, l, off);
                    if (lane == 0) slse[h] = mu + log2f(l);
                }
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < HEADS / 4; ++c) {
                const float4 ls = *reinterpret_cast<const float4 *>(&slse[4 * c]);
                const int live = nh - 4 * c;       // of these four heads; the others' scores are not looked at
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    const float w0 = live > 0 ? fex2(z[k][c].x - ls.x) : 0.f, w1 = live > 1 ? fex2(z[k][c].y - ls.y) : 0.f,
                                w2 = live > 2 ? fex2(z[k][c].z - ls.z) : 0.f, w3 = live > 3 ? fex2(z[k][c].w - ls.w) : 0.f;
                    add[k] += ((w0 + w1) + w2) + w3;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (t0 + tid + k * FIN_THREADS < L) W[k * FIN_THREADS] = sum[k] + add[k];
    };
    using yes = std::true_type;
    using no = std::false_type;
    const bool full = t0 + ACC_TOKENS <= Tcap;
    if (htiles == 1)
        full ? run(yes{}, yes{}) : run(no{}, yes{});
    else
        full ? run(yes{}, no{}) : run(no{}, no{});
}

template <int D, bool Q8, bool RHO, int NT, typename Tout>
cudaError_t launch_t(const DecodeCacheArgs &A, const DecodeCacheScratch &sc, void *mem, const DeviceCtl &ctl,
                     cudaStream_t s) {
    using S = Shape<D, Q8, RHO, NT>;
    const int htiles = (A.pg.group + S::HEADS - 1) / S::HEADS;
    const int Tcap = A.pg.max_pages << A.pg.pshift;
    char *at = static_cast<char *>(mem);
    auto take = [&](size_t n) {
        char *p = n ? at : nullptr;
        at += n;
        return p;
    };
    Scratch ws;
    ws.parts = reinterpret_cast<float *>(take(sc.parts));
    ws.hdr = reinterpret_cast<float4 *>(take(sc.hdr));
    ws.cut = reinterpret_cast<int2 *>(take(sc.cut));
    ws.item = reinterpret_cast<int2 *>(take(sc.item));
    ws.lse2 = reinterpret_cast<float *>(take(sc.lse2));
    ws.zs = reinterpret_cast<float *>(take(sc.zs));
    const bool whole = sc.split != Split::RANGES;
    const int items = A.B * A.pg.Hkv * htiles;
    const int grid = !whole ? sc.ctas : (sc.split == Split::WARPS ? (items + WARPS - 1) / WARPS : items);
    static std::atomic<unsigned long long> limit_set{0};
    if (cudaError_t e = ensure_smem_limit(k_decode_cache<D, Q8, RHO, NT, Tout>, S::SMEM, limit_set)) return e;
    k_decode_cache<D, Q8, RHO, NT, Tout><<<grid, WARPS * 32, S::SMEM, s>>>(
        A.tmk, A.tmv, (const __nv_bfloat16 *)A.q, (const __nv_bfloat16 *)A.rho, A.kexp, A.vexp, A.seqlens, (Tout *)A.y, A.lse, A.B, A.Hq, htiles, sc.split, A.pg, ws, ctl);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (whole && A.wacc == nullptr)) return e;
    // Few items have many parts each and take a block per head, many items have two or three and
    // take one for all heads.  us, a block per head / per item: 8 items of 4096 tokens 14.5 / 18.7,
    // 32 of 8192 26.8 / 28.3, 128 of 4096 39.1 / 39.5 (8 heads each 47.5 / 46.5), 256 of 4096
    // 59.9 / 57.7, 512 of 4096 105.2 / 99.3.
    const int hpb = items >= 128 ? S::HEADS : 1;
    const int combine = whole ? 0 : (hpb == 1 ? items * S::HEADS : grid);
    const int acc_chunks = A.wacc ? (Tcap + ACC_TOKENS - 1) / ACC_TOKENS : 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(combine + (long)A.B * A.pg.Hkv * acc_chunks));
    cfg.blockDim = dim3(FIN_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_decode_finish<D, RHO, S::HEADS, Tout>, ws, A.seqlens, (Tout *)A.y, A.lse, A.wacc,
                              A.Hq, A.pg.Hkv, htiles, Tcap, whole ? 1 : sc.ctas, hpb, combine, Divisor(acc_chunks),
                              Divisor(A.pg.Hkv));
}

template <int D, bool Q8, typename Tout>
cudaError_t launch_d(const DecodeCacheArgs &A, const DecodeCacheScratch &sc, void *mem, const DeviceCtl &ctl,
                     cudaStream_t s) {
    if (A.rho == nullptr) return launch_t<D, Q8, false, 1, Tout>(A, sc, mem, ctl, s);
    if (A.pg.group <= 4) return launch_t<D, Q8, true, 1, Tout>(A, sc, mem, ctl, s);
    return launch_t<D, Q8, true, 2, Tout>(A, sc, mem, ctl, s);
}

template <int D, typename Tout>
cudaError_t launch_q(const DecodeCacheArgs &A, const DecodeCacheScratch &sc, void *mem, const DeviceCtl &ctl,
                     cudaStream_t s) {
    return A.kexp ? launch_d<D, true, Tout>(A, sc, mem, ctl, s) : launch_d<D, false, Tout>(A, sc, mem, ctl, s);
}

// How the work is split, by the table's tokens, the items and the CTAs that are resident.
// us measured, 32 on 8 heads, d = 128, e4m3, half to full tables (*: 0 to full).
//   A warp per item (no merge at all, four times the items under way): 512 items of 256
//   tokens 14.4 against 16.5 with a CTA each, 1024 of 512 28.8 / 34.5, 4096 of 128 33 / 61,
//   8192 of 64 41 / 105; but 512 of 512 22.6 / 21.5, 128 of 128 10.3 / 8.3, and with weights
//   in bf16 512 of 256 22.6 / 18.6*, 1024 of 512 45 / 58*, 4096 of 128 49 / 72*.
//   A CTA per item (no cuts and, but for weights, no second launch) against equal ranges:
//   32 items of 512 10.3 / 12.4, with weights 16 12.9 / 12.2*, bf16 14.5 / 11.1*; without
//   weights 128 items of 1024 14.4 / 18.7, 32 14.4 / 12.4, with weights 96 18.4 / 15.7*;
//   2048 items of 2048 139 / 143, with weights 125 / 152*, bf16 194 / 220*; 512 52 / 49.
Split split_of(size_t items, size_t tokens, size_t ctas, bool q8, bool weights) {
    if ((tokens <= 256 && items >= (q8 ? 1 : 2) * ctas) || (tokens <= 512 && items >= 2 * ctas)) return Split::WARPS;
    if (tokens <= (q8 ? 512u : 256u) || (tokens <= 1024 && items >= 96 && q8 && !weights) ||
        (tokens <= 2048 && items >= 4 * ctas))
        return Split::CTAS;
    return Split::RANGES;
}

}  // namespace

DecodeCacheScratch decode_cache_scratch(const DecodeCacheArgs &A, int sm_count) {
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    const bool rho = A.rho != nullptr, q8 = A.kexp != nullptr;
    const int heads = rho && A.pg.group <= 4 ? 4 : 8;
    const size_t htiles = (A.pg.group + heads - 1) / heads, items = (size_t)A.B * A.pg.Hkv * htiles;
    const size_t cap = (size_t)A.pg.max_pages << A.pg.pshift;
    DecodeCacheScratch s{};
    const bool two = rho && A.pg.group > 4;      // as Shape::CTAS
    const int ctas = sm_count * (two && A.d == 128 ? 2 : (!two && q8 && A.d == 64 ? 4 : 3));
    s.split = split_of(items, cap, ctas, q8, A.wacc != nullptr);
    s.ctas = s.split == Split::RANGES ? ctas : 0;
    s.parts = up((size_t)2 * s.ctas * heads * (rho ? 2 : 1) * A.d * sizeof(float));
    s.hdr = up((size_t)2 * s.ctas * heads * sizeof(float4));
    s.cut = up((size_t)s.ctas * sizeof(int2));
    s.item = s.ctas || A.wacc ? up(items * sizeof(int2)) : 0;
    if (A.wacc) {
        s.lse2 = up((size_t)A.B * A.Hq * sizeof(float));
        s.zs = items * cap * heads * sizeof(float);
    }
    return s;
}

cudaError_t launch_decode_cache(const DecodeCacheArgs &A, const DecodeCacheScratch &sc, void *mem, const DeviceCtl &ctl,
                                cudaStream_t s) {
    if (A.d == 64)
        return A.out_dtype == PARALLAX_F32 ? launch_q<64, float>(A, sc, mem, ctl, s)
                                           : launch_q<64, __nv_bfloat16>(A, sc, mem, ctl, s);
    return A.out_dtype == PARALLAX_F32 ? launch_q<128, float>(A, sc, mem, ctl, s)
                                       : launch_q<128, __nv_bfloat16>(A, sc, mem, ctl, s);
}

}  // namespace plx
