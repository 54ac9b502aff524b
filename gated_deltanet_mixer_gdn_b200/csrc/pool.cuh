// Moves of whole pool rows (a row's recurrent state and its conv history): copy, fork, in-place
// reordering and clearing, each byte read once per distinct source and written once per destination.
//
// The pairs (source, destination) are grouped on the host into sets linked by a shared row.  A task is
// one byte range of one set: the range of every distinct source is loaded into shared memory (bulk
// copies), and only when all have landed is it stored to the destinations.  No other task touches these
// bytes (sets share no rows, tasks of a set share no ranges), so a set may overwrite its own sources --
// a cycle, a swap, beams drawn from one another -- in one launch and without a second buffer.
// The data moves by the bulk-copy engine alone: it never passes through registers.  Bound: HBM.
#pragma once

#include "common.cuh"

namespace gdn {
namespace pool {

constexpr int kMaxOps = 512;             // destinations per launch (the tables are kernel parameters)
constexpr uint32_t kStageBytes = 32768;  // shared memory of one task
// Two CTAs per SM with two stages each: 19 MB on their way over the device.  More in flight only scatters HBM's
// accesses: 128 rows reordered (620 MB) take 101 us so, 106 us with three stages, 110 us with one CTA of six.
constexpr int kStages = 2, kCtasPerSm = 2;
constexpr int kZero = -1;                // source index of a cleared row
constexpr uint32_t kZeroBytes = 4096;
constexpr uint32_t SMEM_BYTES = kStages * kStageBytes + kZeroBytes + 64 + 128;

struct Set {
    int32_t task0;       // first task of the set
    uint16_t src0, nsrc; // its distinct sources in Params::src
    uint16_t op0, nop;   // its destinations in Params::op
    uint32_t chunk;      // bytes of a row per task (multiple of 16)
};
struct Op {
    int32_t dst;         // pool row
    int32_t src;         // index into the set's sources, or kZero
};
struct Params {
    uint8_t* base[2];       // state pool, history pool
    uint32_t row_bytes[2];  // bytes of a row in each
    int32_t nset, ntask, pool_rows;
    Set set[kMaxOps];
    int32_t src[kMaxOps];
    Op op[kMaxOps];
};
static_assert(sizeof(Params) <= 32000, "kernel parameter space");

}  // namespace pool

// One warp per CTA walks the tasks blockIdx.x, blockIdx.x + gridDim.x, ... with kStages of them in
// flight; the lanes share a task's loads and stores.
__global__ void __launch_bounds__(32) gdn_pool_kernel(const __grid_constant__ pool::Params p) {
    using namespace pool;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    uint8_t* zero = smem + kStages * kStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(zero + kZeroBytes);
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
    }
    for (uint32_t i = lane; i < kZeroBytes / 16; i += 32) reinterpret_cast<uint4*>(zero)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
    grid_wait();

    // task -> its set, the pool, the range of the row
    struct Task {
        int set;
        int pool;
        uint32_t off, len;
    };
    auto locate = [&](int t) {
        int lo = 0, hi = p.nset - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.set[mid].task0 <= t) lo = mid;
            else hi = mid - 1;
        }
        Task k;
        k.set = lo;
        const uint32_t c = p.set[lo].chunk;
        uint32_t i = t - p.set[lo].task0;
        const uint32_t n0 = (p.row_bytes[0] + c - 1) / c;
        k.pool = i < n0 ? 0 : 1;
        if (k.pool) i -= n0;
        k.off = i * c;
        k.len = min(c, p.row_bytes[k.pool] - k.off);
        return k;
    };
    auto load = [&](const Task& k, int s) {
        const Set& e = p.set[k.set];
        if (e.nsrc == 0) return;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], k.len * e.nsrc);
        __syncwarp();
        for (int i = lane; i < e.nsrc; i += 32) {
            const int row = p.src[e.src0 + i];
            if (!GDN_CHECK(row >= 0 && row < p.pool_rows)) continue;
            bulk_load(smem + s * kStageBytes + i * e.chunk, p.base[k.pool] + (size_t)row * p.row_bytes[k.pool] + k.off,
                      k.len, &full[s]);
        }
    };
    auto store = [&](const Task& k, int s) {
        const Set& e = p.set[k.set];
        for (int i = lane; i < e.nop; i += 32) {
            const Op o = p.op[e.op0 + i];
            if (!GDN_CHECK(o.dst >= 0 && o.dst < p.pool_rows)) continue;
            uint8_t* dst = p.base[k.pool] + (size_t)o.dst * p.row_bytes[k.pool] + k.off;
            if (o.src != kZero) {
                bulk_store(dst, smem + s * kStageBytes + o.src * e.chunk, k.len);
            } else {
                for (uint32_t b = 0; b < k.len; b += kZeroBytes) bulk_store(dst + b, zero, min(kZeroBytes, k.len - b));
            }
        }
        bulk_commit();
    };

    // the q-th task of this CTA uses stage q % kStages
    const int mine = (p.ntask - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    uint32_t parity = 0;  // bit s: parity of the next phase of full[s]
    bool broken = false;
    int issued = min(kStages, mine);
    for (int q = 0; q < issued; ++q) load(locate(blockIdx.x + q * gridDim.x), q);
    for (int q = 0; q < mine && !broken; ++q) {
        const int s = q % kStages;
        const Task k = locate(blockIdx.x + q * gridDim.x);
        if (p.set[k.set].nsrc != 0) {
            if (!mbar_wait(&full[s], (parity >> s) & 1)) {
                broken = true;
                record_error(kErrTimeoutTma);
                for (int r = q + 1; r < issued; ++r)  // no copy is in flight when the CTA exits
                    if (p.set[locate(blockIdx.x + r * gridDim.x).set].nsrc != 0)
                        mbar_wait(&full[r % kStages], (parity >> (r % kStages)) & 1);
                break;
            }
            parity ^= 1u << s;
        }
        store(k, s);
        // refill the stage of the previous task, whose stores have had this task's wait to read it
        if (q >= 1 && issued < mine) {
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            __syncwarp();
            load(locate(blockIdx.x + issued * gridDim.x), issued % kStages);
            ++issued;
        }
    }
    bulk_wait_all();  // shared memory is read until then
}

}  // namespace gdn
