// Slots sorted by expert in one launch: the maps of the sort (expert_offsets,
// a_map, c_map; rows of an expert in ascending slot order) without its virtual
// experts, for up to 32768 slots.  Longer batches take the sort's three
// launches, which use more than eight SMs.
//
// One CTA, or a cluster of eight, of 32 warps; a warp owns a run of slots, whose
// experts stay in registers.  Count: equal experts of 32 slots are found by
// ballots, the first lane of a group adds its size to the warp's histogram.
// Then an expert's counts become prefixes over the warps of a CTA, over the
// CTAs (each reads the others' totals from their shared memory) and over the
// experts; and the same walk over the slots gives each its row.  Nothing
// depends on timing.
#include <cooperative_groups.h>

#include <algorithm>

#include "route_sort.cuh"
#include "train.cuh"

namespace cg = cooperative_groups;

namespace moe {

namespace {

constexpr int kMapThreads = 1024, kMapWarps = 32, kMapCtas = 8;
constexpr int kMapRounds = 4;    // of 32 slots: a warp's longest run
constexpr int kMapAlone = 2048;  // slots that one CTA sorts

// ROUNDS * 32 slots per warp at most; p.Et <= 1024.
template <int ROUNDS>
__global__ void __launch_bounds__(kMapThreads, 1) token_map_kernel(SortParams p, int rounds) {
    extern __shared__ uint16_t s_count[];  // [warps][Et]: a warp's counts, then the rows before its own in the CTA
    __shared__ int s_total[1024], s_base[1024], s_scan[kMapWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks()), cta = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = p.T * p.kp;
    const int run = rounds * 32, s0 = (cta * kMapWarps + warp) * run;
    uint16_t* mine = s_count + warp * p.Et;

    int e[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int s = s0 + 32 * r + lane;
        e[r] = r < rounds && s < n ? rs::local_expert(p.ids[s], p) : -1;
    }
    for (int x = lane; x < p.Et; x += 32) mine[x] = 0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        if (r >= rounds) break;
        const uint32_t peers = rs::same_expert_lanes(e[r]);
        if (e[r] >= 0 && lane == __ffs(peers) - 1) mine[e[r]] += static_cast<uint16_t>(__popc(peers));
        __syncwarp();
    }
    __syncthreads();
    int total = 0;
    if (tid < p.Et) {
#pragma unroll 8
        for (int w = 0; w < kMapWarps; ++w) {
            const int c = s_count[w * p.Et + tid];
            s_count[w * p.Et + tid] = static_cast<uint16_t>(total);
            total += c;
        }
        s_total[tid] = total;
    }
    cluster.sync();
    int before = 0;  // of this expert in earlier CTAs
    if (ctas > 1 && tid < p.Et) {
        total = 0;
        for (int c = 0; c < ctas; ++c) {
            const int v = cluster.map_shared_rank(s_total, c)[tid];
            if (c < cta) before += v;
            total += v;
        }
    }
    // prefix over the experts, one per thread
    int upto = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    int earlier = lane < warp ? s_scan[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) earlier += __shfl_xor_sync(0xffffffffu, earlier, o);
    upto += earlier;
    if (tid < p.Et) {
        s_base[tid] = upto - total + before;
        if (cta == 0) {
            p.offsets[tid] = upto - total;
            if (tid == p.Et - 1) p.offsets[p.Et] = upto;
        }
    }
    cluster.sync();  // s_base is written; and no CTA leaves while another reads its totals
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        if (r >= rounds) break;
        const int s = s0 + 32 * r + lane;
        const uint32_t peers = rs::same_expert_lanes(e[r]);
        int row = -1;
        if (e[r] >= 0) {
            row = s_base[e[r]] + mine[e[r]] + __popc(peers & ptx::lanemask_lt());
            p.a_map[row] = s;
        }
        if (s < n) p.c_map[s] = row;
        __syncwarp();
        if (e[r] >= 0 && lane == __ffs(peers) - 1) mine[e[r]] += static_cast<uint16_t>(__popc(peers));
        __syncwarp();
    }
}

}  // namespace

cudaError_t launch_token_map(const SortParams& p, cudaStream_t st) {
    const int n = p.T * p.kp;
    if (n > kMapCtas * kMapWarps * kMapRounds * 32) return launch_sort(p, st, false);
    const int ctas = n <= kMapAlone ? 1 : kMapCtas;
    const int rounds = std::max(1, (n + ctas * kMapWarps * 32 - 1) / (ctas * kMapWarps * 32));
    const size_t smem = static_cast<size_t>(kMapWarps) * p.Et * sizeof(uint16_t);  // at most 64 KB
    auto go = [&](auto kernel) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(kMapThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kernel, p, rounds);
    };
    if (rounds <= 2) return go(token_map_kernel<2>);
    return go(token_map_kernel<kMapRounds>);
}

}  // namespace moe
