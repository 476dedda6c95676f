// decode_sched.h -- how the cache decode cuts its work (no CUDA types, so that a
// plain C++ compiler can check it).
//
// An item is one (sequence, KV head, tile of its query heads); its work is the
// sequence's quads (one tile of 16 or 32 tokens for each of a CTA's four warps).
// All items' quads in a row are cut into equal ranges, one per CTA, whatever the
// lengths: the lengths are read on the device, so a ragged batch, one long
// sequence and a table far larger than the sequences all fill the machine.  A
// range covers whole items, whose CTA writes their results, and at most two cut
// ones: the item it starts inside (slot 2 c) and the item it starts but does not
// finish (slot 2 c + 1).  An item cut over CTAs c0 .. c1 has its parts in slots
// 2 c0 + 1, 2 (c0 + 1), .., 2 c1.
#pragma once

#if defined(__CUDACC__)
#define PLX_HD __host__ __device__ __forceinline__
#else
#define PLX_HD inline
#endif

namespace plx {

PLX_HD int quads_of(int tokens, int quad) { return (tokens + quad - 1) / quad; }

// CTAs that take part, of `ctas`, for `total` quads: a quad each at least
PLX_HD int sched_ctas(long long total, int ctas) { return total < ctas ? (int)total : ctas; }
// a / b, in 32 bits where they suffice (a 64-bit division takes the GPU some hundred cycles)
PLX_HD long long sched_div(long long a, long long b) {
    return a <= 0x7fffffff && b <= 0x7fffffff ? (long long)((unsigned)a / (unsigned)b) : a / b;
}
// first quad of CTA c's range
PLX_HD long long sched_start(int c, long long total, int n) { return sched_div((long long)c * total, n); }
// the CTA whose range holds quad x
PLX_HD int sched_owner(long long x, long long total, int n) { return (int)sched_div((x + 1) * n - 1, total); }
// slot of the part of an item that CTA c holds
PLX_HD int sched_slot(int c, bool from_start) { return 2 * c + (from_start ? 1 : 0); }
// slot of part i of an item whose first CTA is c0
PLX_HD int sched_part(int c0, int i) { return i == 0 ? 2 * c0 + 1 : 2 * (c0 + i); }

}  // namespace plx
