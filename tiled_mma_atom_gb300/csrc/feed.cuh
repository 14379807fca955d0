// feed.cuh — how the CTA pairs of the grouped kernels get their tiles.
//
// Tiles have unequal costs (groups of unequal sizes), so a fixed round robin
// leaves pairs idle: simulated over router-like group sizes, 4 to 15 % (64
// groups, 8191 tokens) up to 47 % (128 groups, 3000 tokens, few tiles a group)
// above the mean load, against 1 to 4 % and 20 % when each pair takes the next
// tile as it gets free.  So after its share of the split tiles and its first
// whole tile (both fixed), a pair takes tiles off a counter in global memory.
// Tiles keep their order, and with it the reuse of operands in L2; which pair
// computes a tile does not change its value.
//
// Warp 10 of CTA 0 fetches one tile ahead of the pair's producer, no more: pairs
// start up to 40 us apart when launches overlap, and the first to start would
// take the tiles of the last.  It sends the number to both CTAs with st.async,
// which counts its bytes on the receiver's barrier; warp 10 of each CTA arms
// that barrier.  The warps that read a slot (19 over the pair) free it
// by arriving on CTA 0.  The pair that fetches the last number resets the
// counter, so it is zero again for the next launch.
#pragma once

#include "device.cuh"

namespace tmg {

// A kernel that has given up leaves shared memory and TMEM only when its loads have
// landed and its MMAs have run: wait for the last n uses of the ring before (stage,
// phase), whatever the abort flag says, with a limit of a second at least.  Out of
// line: no call reaches it unless a wait ran out, and its code would cost the others
// (0.3 us of 7.7 at 16 x 4096 x 4096).
static __device__ __noinline__ void settle(uint64_t *bars, int stages, int stage, uint32_t phase, int n, uint32_t *error,
                                           uint64_t budget_ns)
{
    const ErrCtx last{error, budget_ns > 1000000000ull ? budget_ns : 1000000000ull};
    for (int i = 0; i < n && i < stages; ++i) {
        const int s = stage - 1 - i;
        if (!mbar_wait_cluster(&bars[s < 0 ? s + stages : s], s < 0 ? phase ^ 1u : phase, last, nullptr, kSiteDrain))
            return;
    }
}

constexpr int kFeedSlots = 2;
constexpr int kFeedReaders = 19;        // producer and eight epilogue warps of both CTAs, the MMA warp

struct FeedSmem {
    uint64_t full[kFeedSlots], empty[kFeedSlots];
    uint64_t taken;                   // CTA 0: its producer has taken a tile
    int tile[kFeedSlots];
};

__device__ __forceinline__ void feed_init(FeedSmem *f, int readers = kFeedReaders)
{
    for (int i = 0; i < kFeedSlots; ++i) {
        mbar_init(&f->full[i], 1);
        mbar_init(&f->empty[i], readers);
    }
    mbar_init(&f->taken, 1);
}

__device__ __forceinline__ void st_async_u32(uint32_t addr, uint32_t v, uint32_t bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(addr), "r"(v), "r"(bar)
                 : "memory");
}

// Warp 10.  whole: number of whole tiles, handed out from `nclusters` on.
__device__ __forceinline__ void feed_run(FeedSmem *f, uint32_t rank, int whole, int nclusters, uint32_t *counter,
                                         const ErrCtx &err, volatile int *abort)
{
    if (whole <= nclusters)
        return;
    const uint32_t last = static_cast<uint32_t>(whole - nclusters) + static_cast<uint32_t>(nclusters) - 1;
    int slot = 0;
    uint32_t phase = 0;
    for (uint32_t n = 0;; ++n) {
        int tile = 0;
        if (rank == 0) {
            if (n > 0 && !mbar_wait_warp(&f->taken, (n - 1) & 1u, err, abort, kSiteProducerEmpty))
                return;
            if (!mbar_wait_cluster_warp(&f->empty[slot], phase ^ 1u, err, abort, kSiteProducerEmpty))
                return;
            uint32_t v = 0;
            if ((threadIdx.x & 31) == 0) {
                v = atomicAdd(counter, 1u);
                if (v == last)
                    *counter = 0;
            }
            v = __shfl_sync(0xffffffffu, v, 0);
            tile = nclusters + static_cast<int>(v);
        }
        mbar_arrive_expect_tx_w(&f->full[slot], 4);
        if (rank == 0 && (threadIdx.x & 31) < 2) {
            const uint32_t to = threadIdx.x & 31;
            st_async_u32(mapa_shared(smem_u32(&f->tile[slot]), to), static_cast<uint32_t>(tile),
                         mapa_shared(smem_u32(&f->full[slot]), to));
        }
        __syncwarp();
        // CTA 1 learns here when to stop; CTA 0 leaves only after its own copy
        // has landed
        if (!mbar_wait_cluster_warp(&f->full[slot], phase, err, abort, kSiteProducerEmpty))
            return;
        tile = *const_cast<volatile int *>(&f->tile[slot]);
        if (tile >= whole)
            return;
        if (++slot == kFeedSlots) {
            slot = 0;
            phase ^= 1u;
        }
    }
}

// A reading warp's view: the whole tiles of its pair, in order.
struct Feed {
    FeedSmem *f;
    int whole, nclusters, first;      // first: the pair's fixed tile, or -1 once taken
    int slot = 0;
    uint32_t phase = 0;
    bool producer = false;            // CTA 0's producer

    __device__ Feed(FeedSmem *f_, int cluster, int nclusters_, int whole_)
        : f(f_), whole(whole_), nclusters(nclusters_), first(cluster)
    {
    }

    __device__ __forceinline__ bool next(int &tile, const ErrCtx &err, volatile int *abort)
    {
        if (first >= 0) {
            tile = first;
            first = -1;
            return tile < whole;
        }
        if (whole <= nclusters)
            return false;
        if (!mbar_wait_cluster_warp(&f->full[slot], phase, err, abort, kSiteMmaFull))
            return false;
        tile = *const_cast<volatile int *>(&f->tile[slot]);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            mbar_arrive_cluster(mapa_shared(smem_u32(&f->empty[slot]), 0));
            if (producer)
                mbar_arrive_cluster(smem_u32(&f->taken));
        }
        if (++slot == kFeedSlots) {
            slot = 0;
            phase ^= 1u;
        }
        return tile < whole;
    }
};

}  // namespace tmg
