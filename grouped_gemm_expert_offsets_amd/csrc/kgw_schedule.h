// Which output tiles a workgroup of the persistent weight-gradient kernels computes, and each tile's token range.
#pragma once

#include "kgw_device.h"
#include "kgw_internal.h"

namespace kgw {

// Static schedule: round r covers items [r*G, (r+1)*G); with p.snake the slots of odd
// rounds run in reverse, so a workgroup alternates between the front and the back of
// consecutive rounds (each XCD still holds a contiguous run of items).
//
// Dynamic schedule (p.sched): the same runs of G/nq items per round form nq queues, one
// per XCD (queue q: the q-th run of every round), claimed one item at a time through
// the queue's counter; a workgroup drains the queue of its XCD (block id mod nq, the
// hardware's round-robin placement), then those of the next ones, so every claimed
// index is unique and every workgroup stops after at most nq empty claims.  Experts
// run longest first: lane k of every wave holds the expert of rank k (ties by index),
// so the last items to be claimed are the shortest.  Thread 0 claims the next item
// while the current one writes its output, and passes it on through LDS word 0 (the
// rings are idle between items) between two barriers.  The barriers order nothing by
// themselves: the word is waited for before the first (or others could read what was there,
// part of the last tile, and take it for an item) and each wave's read before the second
// (or the next item's ring could overwrite it).
struct Schedule {
    const GroupedParams& p;
    lds_char* const tiles;
    const int tid, G, slot, nq, qrun;
    const bool dyn;
    int perm;               // dynamic: the expert of this lane's rank
    int q, left;            // thread 0's queue state
    int r = 0;              // static: next round
    int pend = 0;           // thread 0: raw claim of the next item

    __device__ __forceinline__ Schedule(const GroupedParams& p_, lds_char* tiles_, int tid_)
        : p(p_), tiles(tiles_), tid(tid_), G(gridDim.x), slot(xcd_slot(blockIdx.x, gridDim.x, p_.num_xcds)),
          nq(p_.num_xcds), qrun((int)gridDim.x / p_.num_xcds), dyn(p_.sched != nullptr), perm(tid_ & 63),
          q((int)(blockIdx.x % (unsigned)p_.num_xcds)), left(p_.num_xcds) {
        if (!dyn) return;
        const int lane = tid & 63, E = p.num_experts;       // <= kSchedMaxExperts
        const int64_t T = p.tokens_sum;
        int cnt = -1;
        if (lane < E) {
            const int64_t b0 = lane ? (int64_t)p.offsets[lane - 1] : 0, e0 = p.offsets[lane];
            const int64_t b1 = b0 < 0 ? 0 : (b0 > T ? T : b0);
            const int64_t e1 = e0 < 0 ? 0 : (e0 > T ? T : e0);
            cnt = (int)(e1 > b1 ? e1 - b1 : 0);
        }
        int rank = lane;
        if (lane < E) {
            rank = 0;
            for (int j = 0; j < E; ++j) {
                const int cj = __builtin_amdgcn_readlane(cnt, j);
                rank += (cj > cnt || (cj == cnt && j < lane)) ? 1 : 0;
            }
        }
        perm = __builtin_amdgcn_ds_permute(rank << 2, lane);
        if (tid == 0) pend = atomicAdd(p.sched + q, 1);
    }

    // thread 0: the item of raw claim `idx` in queue q; an exhausted queue sends it on to
    // the next one (claiming there), -1 once every queue is exhausted
    __device__ __forceinline__ int resolve(int idx) {
        for (;;) {
            const int it = (idx / qrun) * G + q * qrun + idx % qrun;
            if (it < p.num_items) return it;
            if (--left == 0) return -1;
            q = q + 1 == nq ? 0 : q + 1;
            idx = atomicAdd(p.sched + q, 1);
        }
    }
    __device__ __forceinline__ int broadcast(int v) {
        if (tid == 0) *(__attribute__((address_space(3))) int*)tiles = v;
        asm volatile("" ::: "memory");
        wait_lgkmcnt0();
        barrier_no_fence();
        v = *(__attribute__((address_space(3))) int*)tiles;
        asm volatile("" ::: "memory");
        wait_lgkmcnt0();
        barrier_no_fence();
        return __builtin_amdgcn_readfirstlane(v);
    }
    __device__ __forceinline__ int next_static() {
        while (r * G < p.num_items) {
            const int it = r * G + ((r & 1) && p.snake ? G - 1 - slot : slot);
            ++r;
            if (it < p.num_items) return it;
        }
        return -1;
    }
    __device__ __forceinline__ void claim_next() {
        if (dyn && tid == 0) pend = atomicAdd(p.sched + q, 1);
    }
    // The next item, -1 past the last.  With a static schedule no waves meet here.
    __device__ __forceinline__ int next() {
        if (!dyn) return next_static();
        return broadcast(tid == 0 ? resolve(pend) : 0);
    }
    // Expert of the item with expert slot `ec` (expert-major, p.split chunks each).
    __device__ __forceinline__ int expert(int ec) const {
        return dyn ? __builtin_amdgcn_readlane(perm, ec) : ec / p.split;   // dynamic: split is 1
    }
};

// Tokens [ebegin, eend) of expert e, clamped into [0, T), and those [begin, end) of its K chunk c.
struct TokenRange {
    int32_t ebegin, eend, begin, end;
};
__device__ __forceinline__ TokenRange token_range(const GroupedParams& p, int e, int c) {
    const int64_t T = p.tokens_sum;
    const int64_t raw_begin = e ? (int64_t)p.offsets[e - 1] : 0;
    const int64_t raw_end = p.offsets[e];
    TokenRange t;
    t.ebegin = (int32_t)(raw_begin < 0 ? 0 : (raw_begin > T ? T : raw_begin));
    t.eend = max(t.ebegin, (int32_t)(raw_end < 0 ? 0 : (raw_end > T ? T : raw_end)));
    t.begin = t.ebegin;
    t.end = t.eend;
    if (p.split > 1) {
        const int32_t len = ((t.end - t.begin + p.split - 1) / p.split + kSplitUnit - 1) & ~(kSplitUnit - 1);
        const int32_t cb = (int32_t)min<int64_t>(t.end, (int64_t)t.begin + (int64_t)c * len);
        t.end = (int32_t)min<int64_t>(t.end, (int64_t)cb + len);
        t.begin = cb;
    }
    return t;
}

}  // namespace kgw
