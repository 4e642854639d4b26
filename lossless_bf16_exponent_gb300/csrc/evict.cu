// evict.cu -- eviction from a cache by accumulated attention weight: select
// the tokens to keep of each sequence and KV head, and pack their keys and
// values in a contiguous buffer.
//
// Select: the keep-th largest mass is found by radix selection on 32-bit keys
// whose order is the masses' (protected slots above every number, NaN below),
// eight bits a pass, until the keys of the threshold's bin are all kept or all
// bits are decided. Of keys equal to the threshold the lowest slots are kept.
// One thread-block cluster takes one row (sequence, KV head), each of its CTAs
// a contiguous share of the slots, whose keys it holds in shared memory (rows
// beyond eight shares of kCached slots are read again each pass). A pass is
// one barrier: counts, summed over the cluster through distributed shared
// memory, then every warp finds the threshold's digit by itself. Bound: latency,
// a few microseconds of barriers and shared-memory rounds. Kept slots
// are written in slot order: a warp owns consecutive slots, 32 a step, so that
// ballots give each kept slot its place within the warp's.
//
// Pack: bound by HBM; each kept row is read and written once, 16 bytes a lane.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "kv_internal.cuh"

namespace cg = cooperative_groups;

namespace uzkv {
namespace {

constexpr uint32_t kCached = 32768;  // keys of a CTA's share in shared memory
constexpr int kPackThreads = 256;

struct Params {
    Cache cache;
    const float* mass;
    int64_t mass_b, mass_h;  // elements
    uint32_t slots, keep, sink, recent;
    Rows out_k, out_v;
    int32_t* kept;
    float* mass_out;
    int32_t* lengths_out;
    uint32_t row_chunks;  // 16-byte chunks of a row
};

__device__ __forceinline__ uint32_t key_of(float x, uint32_t slot, uint32_t len, const Params& p) {
    if (slot < p.sink || slot + p.recent >= len) return 0xFFFFFFFFu;
    if (x != x) return 0;
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0: the two zeros are equal masses
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ uint32_t row_length(const Params& p, uint32_t b) {
    const Span s = span_of(p.cache, nullptr, 0, b);
    if (s.old > p.slots) corrupt(p.cache);
    return min(s.old, p.slots);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) select_kernel(const __grid_constant__ Params p, uint32_t cached) {
    constexpr int kWarps = THREADS / 32;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ uint32_t keys[];  // [cached] of this CTA's share, if it fits
    __shared__ uint32_t hist[4][256];
    __shared__ uint32_t totals[4][256];
    __shared__ uint32_t sums[2][kWarps];
    __shared__ uint32_t share[2];  // this CTA's keys above and at the threshold
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t row = blockIdx.y, b = row / p.cache.kv_heads, h = row % p.cache.kv_heads;
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    uzip::pdl_launch_dependents();
    const uint32_t len = row_length(p, b);
    const uint32_t target = min(len, p.keep);
    const float* mass = p.mass + b * p.mass_b + h * p.mass_h;
    int32_t* kept = p.kept + (uint64_t)row * p.keep;
    float* mass_out = p.mass_out + (uint64_t)row * p.keep;

    if (h == 0 && rank == 0 && tid == 0) p.lengths_out[b] = (int32_t)target;
    for (uint32_t r = target + rank * THREADS + tid; r < p.keep; r += ranks * THREADS) {
        kept[r] = -1;
        mass_out[r] = 0.0f;
    }
    if (target == len) {  // keeps all (also an empty sequence)
        for (uint32_t j = rank * THREADS + tid; j < len; j += ranks * THREADS) {
            kept[j] = (int32_t)j;
            mass_out[j] = mass[j];
        }
        return;  // the whole cluster returns here
    }

    // This CTA's share, and of it each warp's: whole steps of 32 slots.
    const uint32_t per = ((len + ranks - 1) / ranks + 31) / 32 * 32;
    const uint32_t begin = min(len, rank * per), end = min(len, begin + per);
    const uint32_t seg = (per / 32 + kWarps - 1) / kWarps * 32;
    const uint32_t w0 = min(end, begin + warp * seg), w1 = min(end, w0 + seg);
    const bool held = per <= cached;
    for (uint32_t i = tid; i < 4 * 256; i += THREADS) reinterpret_cast<uint32_t*>(hist)[i] = 0;
    if (held)
#pragma unroll 4
        for (uint32_t j = begin + tid; j < end; j += THREADS) keys[j - begin] = key_of(mass[j], j, len, p);
    __syncthreads();
    auto key_at = [&](uint32_t j) { return held ? keys[j - begin] : key_of(mass[j], j, len, p); };

    // Threshold key: its digits from the top; `want` is how many keys are still to be taken at or below the
    // decided digits. Masses share few leading bits, so lanes with the same first digit add up before they count.
    uint32_t prefix = 0, want = target, threshold = 0;
#pragma unroll 1
    for (int pass = 0; pass < 4; pass++) {
        const uint32_t shift = 24 - 8 * pass;
        if (pass == 0) {
            for (uint32_t j0 = w0; j0 < w1; j0 += 32) {
                const bool in = j0 + lane < w1;
                const uint32_t digit = in ? key_at(j0 + lane) >> 24 : 256;
                const uint32_t same = __match_any_sync(0xFFFFFFFFu, digit);
                if (in && (int)lane == __ffs(same) - 1) atomicAdd(&hist[0][digit], (uint32_t)__popc(same));
            }
        } else {
#pragma unroll 4
            for (uint32_t j = w0 + lane; j < w1; j += 32) {
                const uint32_t key = key_at(j);
                if ((key >> (shift + 8)) == prefix) atomicAdd(&hist[pass][(key >> shift) & 255], 1u);
            }
        }
        const uint32_t* count = hist[pass];
        if (ranks > 1) {
            cluster.sync();
            if (tid < 256) {
                uint32_t n = 0;
                for (uint32_t r = 0; r < ranks; r++) n += cluster.map_shared_rank(&hist[pass][0], r)[tid];
                totals[pass][tid] = n;
            }
            count = totals[pass];
        }
        __syncthreads();
        // Lane l holds digits 255 - 8 l down to 248 - 8 l; the threshold's is where the running count reaches `want`.
        uint32_t mine[8], n = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            mine[i] = count[255 - 8 * lane - i];
            n += mine[i];
        }
        uint32_t upto = n;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= (uint32_t)o) upto += v;
        }
        const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, upto >= want)) - 1;
        uint32_t above = upto - n, digit = 0, at = 0;
        bool found = false;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if (!found && want <= above + mine[i]) {
                found = true;
                digit = 255 - 8 * lane - i;
                at = mine[i];
            }
            if (!found) above += mine[i];
        }
        digit = __shfl_sync(0xFFFFFFFFu, digit, owner);
        want -= __shfl_sync(0xFFFFFFFFu, above, owner);
        at = __shfl_sync(0xFFFFFFFFu, at, owner);
        prefix = prefix << 8 | digit;
        threshold = prefix << shift;
        if (at == want && threshold) {  // all of the bin is kept: every key from its lowest on
            threshold -= 1;
            want = 0;
            break;
        }
    }
    // Keys above the threshold are kept, and the first `want` equal to it.

    uint32_t gt = 0, eq = 0;  // of this warp's slots
    for (uint32_t j0 = w0; j0 < w1; j0 += 32) {
        const uint32_t key = j0 + lane < w1 ? key_at(j0 + lane) : 0;
        gt += __popc(__ballot_sync(0xFFFFFFFFu, j0 + lane < w1 && key > threshold));
        eq += __popc(__ballot_sync(0xFFFFFFFFu, j0 + lane < w1 && key == threshold));
    }
    if (lane == 0) {
        sums[0][warp] = gt;
        sums[1][warp] = eq;
    }
    __syncthreads();
    uint32_t g = lane < kWarps ? sums[0][lane] : 0, e = lane < kWarps ? sums[1][lane] : 0;
    const uint32_t g0 = g, e0 = e;
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, g, o), y = __shfl_up_sync(0xFFFFFFFFu, e, o);
        if (lane >= (uint32_t)o) {
            g += x;
            e += y;
        }
    }
    if (warp == 0 && lane == 31) {
        share[0] = g;
        share[1] = e;
    }
    g = __shfl_sync(0xFFFFFFFFu, g - g0, warp);
    e = __shfl_sync(0xFFFFFFFFu, e - e0, warp);
    if (ranks > 1) {
        cluster.sync();
        for (uint32_t r = 0; r < rank; r++) {
            const uint32_t* s = cluster.map_shared_rank(&share[0], r);
            g += s[0];
            e += s[1];
        }
    }
    for (uint32_t j0 = w0; j0 < w1; j0 += 32) {
        const uint32_t j = j0 + lane, below = (1u << lane) - 1;
        const uint32_t key = j < w1 ? key_at(j) : 0;
        const uint32_t gs = __ballot_sync(0xFFFFFFFFu, j < w1 && key > threshold);
        const uint32_t es = __ballot_sync(0xFFFFFFFFu, j < w1 && key == threshold);
        const uint32_t ge = g + __popc(gs & below), ee = e + __popc(es & below);
        if (j < w1 && (key > threshold || (key == threshold && ee < want))) {
            const uint32_t at = ge + min(ee, want);
            kept[at] = (int32_t)j;
            mass_out[at] = mass[j];
        }
        g += __popc(gs);
        e += __popc(es);
    }
    if (ranks > 1) cluster.sync();  // no CTA leaves while another reads its shared memory
}

__global__ void __launch_bounds__(kPackThreads) pack_kernel(const __grid_constant__ Params p) {
    const uint32_t row = blockIdx.y, b = row / p.cache.kv_heads, h = row % p.cache.kv_heads;
    const uint32_t total = p.keep * p.row_chunks;
    const int32_t* kept = p.kept + (uint64_t)row * p.keep;
    uzip::pdl_wait();
    for (uint32_t i = blockIdx.x * kPackThreads + threadIdx.x; i < total; i += gridDim.x * kPackThreads) {
        const uint32_t r = i / p.row_chunks, c = i % p.row_chunks * 16;
        const int32_t j = kept[r];
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        if (j >= 0) {
            const Place at = place_of(p.cache, b, (uint32_t)j);
            if (at.page >= 0) {
                k = uzip::ld_stream_v4(k_row(p.cache, at, h) + c);
                v = uzip::ld_stream_v4(v_row(p.cache, at, h) + c);
            }
        }
        *reinterpret_cast<uint4*>(p.out_k.p + b * p.out_k.b + h * p.out_k.t + r * p.out_k.h + c) = k;
        *reinterpret_cast<uint4*>(p.out_v.p + b * p.out_v.b + h * p.out_v.t + r * p.out_v.h + c) = v;
    }
}

}  // namespace
}  // namespace uzkv

using namespace uzkv;

extern "C" UZIP_API int uzkv_evict(const uzkv_cache_t* cache, const float* d_mass, int64_t mass_stride_b,
                                   int64_t mass_stride_h, uint32_t slots, uint32_t keep, uint32_t sink,
                                   uint32_t recent, const uzkv_rows_t* out_k, const uzkv_rows_t* out_v,
                                   int32_t* d_kept, float* d_mass_out, int32_t* d_lengths_out, uzip_stream_t stream) {
    Params p{};
    if (int rc = cache_of(cache, &p.cache)) return rc;
    if (!d_mass || !d_kept || !d_mass_out || !d_lengths_out || !rows_valid(out_k) || !rows_valid(out_v)) return UZIP_ERR_ARG;
    if (mass_stride_b < 0 || mass_stride_h < 0 || !slots || slots > 0x7FFFFF00u) return UZIP_ERR_ARG;
    if (!keep || (uint64_t)sink + recent > keep || (uint64_t)keep * 32 > 0xFFFFFFFFull) return UZIP_ERR_ARG;
    if ((uint64_t)p.cache.sequences * p.cache.kv_heads > 65535) return UZIP_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(d_mass) | reinterpret_cast<uintptr_t>(d_kept) |
         reinterpret_cast<uintptr_t>(d_mass_out) | reinterpret_cast<uintptr_t>(d_lengths_out)) & 3)
        return UZIP_ERR_ALIGN;
    p.out_k = rows_of(out_k, cache->dtype);
    p.out_v = rows_of(out_v, cache->dtype);
    if (!rows_aligned16(p.out_k) || !rows_aligned16(p.out_v)) return UZIP_ERR_ALIGN;
    p.mass = d_mass;
    p.mass_b = mass_stride_b;
    p.mass_h = mass_stride_h;
    p.slots = slots;
    p.keep = keep;
    p.sink = sink;
    p.recent = recent;
    p.kept = d_kept;
    p.mass_out = d_mass_out;
    p.lengths_out = d_lengths_out;
    p.row_chunks = p.cache.head_dim * bytes_of(cache->dtype) / 16;
    int sms = 0;
    if (int rc = sm_count(&sms)) return rc;
    const uint32_t rows = p.cache.sequences * p.cache.kv_heads;
    // A row's CTAs: up to eight while the SMs have room and a share keeps 4096 slots.
    uint32_t ranks = 1;
    while (ranks < 8 && rows * ranks * 2 <= (uint32_t)sms && slots / ranks > 4096) ranks *= 2;
    const uint32_t per = ((slots + ranks - 1) / ranks + 31) / 32 * 32, held = per <= kCached ? per : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ranks, rows);
    cfg.stream = s;
    cfg.dynamicSmemBytes = held * 4;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    if (per <= 4096) {  // short shares: fewer warps meet at the barriers
        cfg.blockDim = dim3(256);
        UZIP_CUDA_TRY(cudaLaunchKernelEx(&cfg, select_kernel<256>, p, held));
    } else {
        static std::atomic<uint64_t> ready{0};  // a bit for each device whose limit is raised
        int dev = 0;
        UZIP_CUDA_TRY(cudaGetDevice(&dev));
        if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
            UZIP_CUDA_TRY(cudaFuncSetAttribute(select_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kCached * 4));
            if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
        }
        cfg.blockDim = dim3(1024);
        UZIP_CUDA_TRY(cudaLaunchKernelEx(&cfg, select_kernel<1024>, p, held));
    }
    const uint64_t chunks = (uint64_t)keep * p.row_chunks;
    const uint64_t want = std::max<uint64_t>(1, (uint64_t)sms * 32 / rows);
    const unsigned grid = (unsigned)std::min<uint64_t>((chunks + kPackThreads - 1) / kPackThreads, want);
    cudaLaunchConfig_t pack{};
    pack.gridDim = dim3(grid, rows);
    pack.blockDim = dim3(kPackThreads);
    pack.stream = s;
    cudaLaunchAttribute early[1];  // launched while the selection still runs; waits for it on the device
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    pack.attrs = early;
    pack.numAttrs = 1;
    UZIP_CUDA_TRY(cudaLaunchKernelEx(&pack, pack_kernel, p));
    return UZIP_OK;
}
