// beam_reorder.cu -- the recurrent states of a beam search after a selection (gdn_beam_reorder).
//
// A state is 64 KB per head, so what counts is how few of them move: a parent's first child keeps the
// parent's slot, and only further children are copied, into slots of beams that died. Sources and
// destinations are then different slots, so the copies need no order and no staging. Every CTA works
// out the list of copies for itself (parents and slots are a few KB that stay in L2), then takes
// 16 KB pieces of (copy, pool) in turn. Bound by memory: each copied byte is read and written once.
#include <cstdint>

#include "gdn_beam.h"
#include "gdn_chain.cuh"
#include "gdn_common.cuh"

namespace gdn {

namespace {

constexpr int kReThreads = 256;
constexpr int kReMaxBeams = 2048;           // beams of one launch (the list of copies is in shared memory)
constexpr int64_t kRePiece = 16 * 1024;     // bytes

struct ReorderPool {
    unsigned char *base;
    int64_t stride, bytes;
    int pieces_before;                      // pieces of one slot in the pools before this one
    int width;                              // bytes per access: the largest power of two up to 16 that all addresses allow
};

struct ReorderLaunch {
    const int32_t *slots, *parents;
    int32_t *new_slots, *err_flags;
    int batch, beams, num_slots, num_pools, pieces;
    ReorderPool pool[GDN_BEAM_MAX_POOLS];
};
static_assert(sizeof(ReorderLaunch) <= 4096 + 512, "kernel parameters");

template <typename W> __device__ __forceinline__ void copy_piece(unsigned char *dst, const unsigned char *src, int64_t bytes, int tid)
{
    const int n = (int)(bytes / (int)sizeof(W));
    W *d = reinterpret_cast<W *>(dst);
    const W *s = reinterpret_cast<const W *>(src);
    for (int i0 = 0; i0 < n; i0 += 4 * kReThreads) {
        W v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * kReThreads + tid < n) v[k] = s[i0 + k * kReThreads + tid];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * kReThreads + tid < n) d[i0 + k * kReThreads + tid] = v[k];
    }
}

__global__ void __launch_bounds__(kReThreads) beam_reorder_kernel(const __grid_constant__ ReorderLaunch P)
{
    __shared__ short par[kReMaxBeams];      // parent, or -1
    __shared__ int slot_of[kReMaxBeams];
    __shared__ unsigned char first[kReMaxBeams], kept[kReMaxBeams];
    __shared__ int2 copies[kReMaxBeams];    // source slot, destination slot
    __shared__ int wcount[kReThreads / 32];
    ordinary_launch_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = P.batch * P.beams, beams = P.beams;

    for (int i = tid; i < R; i += kReThreads) {
        const int p = P.parents[i];
        par[i] = p >= 0 && p < beams ? (short)p : (short)-1;
        slot_of[i] = P.slots[i];
        kept[i] = 0;
    }
    __syncthreads();
    for (int i = tid; i < R; i += kReThreads) {
        const int b0 = i - i % beams, p = par[i];
        bool f = p >= 0;
        for (int j = b0; j < i; ++j) f = f && par[j] != p;
        first[i] = f;
        if (f) kept[b0 + p] = 1;            // one first child per parent: no two threads write here
    }
    __syncthreads();
    int total = 0;
    for (int i0 = 0; i0 < R; i0 += kReThreads) {
        const int i = i0 + tid;
        bool copy = false;
        int2 c = make_int2(0, 0);
        if (i < R) {
            const int b0 = i - i % beams, p = par[i];
            int slot;
            if (first[i]) {
                slot = slot_of[b0 + p];
            } else {
                int rank = 0;               // how many before this one need a free slot
                for (int j = b0; j < i; ++j) rank += !first[j];
                int j = b0;
                for (;; ++j)
                    if (!kept[j] && rank-- == 0) break;      // as many are free as are needed
                slot = slot_of[j];
                if (p >= 0) {
                    c = make_int2(slot_of[b0 + p], slot);
                    copy = c.x >= 0 && c.x < P.num_slots && c.y >= 0 && c.y < P.num_slots;
                    if (!copy && blockIdx.x == 0) raise_flag(P.err_flags, GDN_DEVERR_BAD_INDEX);
                }
            }
            if (blockIdx.x == 0) P.new_slots[i] = slot;
        }
        const unsigned vote = __ballot_sync(0xFFFFFFFFu, copy);
        if (lane == 0) wcount[warp] = __popc(vote);
        __syncthreads();
        int at = total + __popc(vote & ((1u << lane) - 1));
        for (int w = 0; w < kReThreads / 32; ++w) {
            if (w < warp) at += wcount[w];
            total += wcount[w];
        }
        if (copy) copies[at] = c;
        __syncthreads();
    }

    const int64_t units = (int64_t)total * P.pieces;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int2 c = copies[(int)(u % total)];
        const int piece = (int)(u / total);
        int lo = 0, hi = P.num_pools - 1;   // the last pool with pieces_before <= piece
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (P.pool[mid].pieces_before <= piece) lo = mid; else hi = mid - 1;
        }
        const ReorderPool &q = P.pool[lo];
        const int64_t off = (int64_t)(piece - q.pieces_before) * kRePiece;
        const int64_t n = min(kRePiece, q.bytes - off);
        if (!GDN_IN(P.err_flags, off, q.bytes) || !GDN_IN(P.err_flags, n - 1, kRePiece)) continue;
        const unsigned char *src = q.base + c.x * q.stride + off;
        unsigned char *dst = q.base + c.y * q.stride + off;
        switch (q.width) {
        case 16: copy_piece<uint4>(dst, src, n, tid); break;
        case 8: copy_piece<uint2>(dst, src, n, tid); break;
        case 4: copy_piece<uint32_t>(dst, src, n, tid); break;
        case 2: copy_piece<uint16_t>(dst, src, n, tid); break;
        default: copy_piece<uint8_t>(dst, src, n, tid); break;
        }
    }
}

bool overlap(const void *p, size_t pn, const void *q, size_t qn)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + qn && b < a + pn;
}

}  // namespace

}  // namespace gdn

extern "C" int gdn_beam_reorder(const gdn_beam_reorder_args *a, gdn_stream_t stream)
{
    using namespace gdn;
    if (!a) return GDN_ERR_NULL;
    if (a->batch < 0 || a->beams < 1 || a->beams > GDN_BEAM_MAX_BEAMS || a->num_slots < 1 || a->num_pools < 0 ||
        a->num_pools > GDN_BEAM_MAX_POOLS)
        return GDN_ERR_SHAPE;
    if ((a->num_pools > 0 && !a->pools) || (a->batch > 0 && (!a->slots || !a->parents || !a->new_slots))) return GDN_ERR_NULL;
    // every CTA reads both tables, and the first writes new_slots while others may still be reading
    const size_t table = (size_t)a->batch * a->beams * sizeof(int32_t);
    if (overlap(a->new_slots, table, a->slots, table) || overlap(a->new_slots, table, a->parents, table)) return GDN_ERR_ARG;
    for (const void *p : {(const void *)a->slots, (const void *)a->parents, (const void *)a->new_slots})
        if (reinterpret_cast<uintptr_t>(p) % 4) return GDN_ERR_ALIGN;
    ReorderLaunch P;
    P.err_flags = a->err_flags;
    P.beams = a->beams;
    P.num_slots = a->num_slots;
    P.num_pools = 0;
    int64_t pieces = 0;
    for (int i = 0; i < a->num_pools; ++i) {
        const gdn_beam_pool &p = a->pools[i];
        if (p.slot_bytes < 0 || p.slot_stride < p.slot_bytes) return GDN_ERR_SHAPE;
        if (p.slot_bytes == 0) continue;
        if (!p.base) return GDN_ERR_NULL;
        ReorderPool &q = P.pool[P.num_pools++];
        q.base = static_cast<unsigned char *>(p.base);
        q.stride = p.slot_stride;
        q.bytes = p.slot_bytes;
        q.pieces_before = (int)pieces;
        q.width = 16;
        while ((reinterpret_cast<uintptr_t>(p.base) | (uintptr_t)p.slot_stride | (uintptr_t)p.slot_bytes) % q.width) q.width /= 2;
        pieces += (p.slot_bytes + kRePiece - 1) / kRePiece;
        if (pieces > INT32_MAX) return GDN_ERR_SHAPE;
    }
    P.pieces = (int)pieces;
    // as many batch entries at a time as the list of copies holds
    const int step = kReMaxBeams / a->beams;
    for (int b = 0; b < a->batch; b += step) {
        P.batch = a->batch - b < step ? a->batch - b : step;
        P.slots = a->slots + (int64_t)b * a->beams;
        P.parents = a->parents + (int64_t)b * a->beams;
        P.new_slots = a->new_slots + (int64_t)b * a->beams;
        const int64_t most = (int64_t)P.batch * (a->beams - 1) * pieces;      // a parent's first child is not copied
        const int64_t ctas = most < 1 ? 1 : most < 152 * 6 ? most : 152 * 6;
        if (launch_ordinary(beam_reorder_kernel, dim3((unsigned)ctas), dim3(kReThreads), 0,
                            reinterpret_cast<cudaStream_t>(stream), P) != cudaSuccess)
            return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}
