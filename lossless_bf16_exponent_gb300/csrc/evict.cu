// evict.cu -- eviction from a cache by accumulated attention weight: select
// the tokens to keep of each sequence and KV head, and pack their keys and
// values in a contiguous buffer.
//
// Select: the keep-th largest mass is found by radix selection on 32-bit keys
// whose order is the masses' (protected slots above every number, NaN below),
// eight bits a pass, until the keys of the threshold's bin are all kept or all
// bits are decided. Of keys equal to the threshold the lowest slots are kept.
// One thread-block cluster takes one row (sequence, KV head), each of its CTAs
// a contiguous share of the slots, whose keys it holds in shared memory (longer
// shares are read again each pass). The second pass lists the keys that share
// the first's digit, and later ones go through that list only. Counts of a
// pass are summed over the cluster through distributed shared memory (the first
// pass's spread over copies: masses share few leading bits). Bound: latency, some microseconds of barriers and shared-
// memory rounds. Kept slots are written in slot order: a warp owns consecutive
// slots, 32 a step, so that ballots give each kept slot its place.
//
// Pack: bound by HBM; each kept row is read and written once, 16 bytes a lane.
//
// Measured: 131,072 slots of 8 heads to 16,384 kept rows of 128: 36 us, 17 of them the selection and 19 the packing of
// 134 MB (7 TB/s); 160 rows of up to 3,001 slots to 500 of 64 bytes: 12 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "kv_index.cuh"
#include "kv_internal.cuh"

namespace cg = cooperative_groups;

namespace uzkv {
namespace {

constexpr uint32_t kCached = 23552;  // keys of a CTA's share in shared memory, and as many of the second pass's list
constexpr uint32_t kMaxRanks = 8;    // CTAs of a row (16 measured slower: the barriers)
constexpr uint32_t kCopies = 32;     // of the first pass's counts, one a lane
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
    extern __shared__ uint32_t keys[];  // [cached] of this CTA's share, if it fits; [cached] list
    __shared__ uint32_t first[kCopies][256 + 1];  // a copy's digits one bank on from the last one's
    __shared__ __align__(16) uint32_t hist[4][256];
    __shared__ __align__(16) uint32_t hist_all[256];  // of the cluster
    __shared__ uint4 choice;
    __shared__ uint32_t sums[2][kWarps];
    __shared__ __align__(8) uint32_t share[2];  // this CTA's keys above and at the threshold
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t row = blockIdx.y, b = row / p.cache.kv_heads, h = row % p.cache.kv_heads;
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    uzip::pdl_launch_dependents();
    const float* mass = p.mass + b * p.mass_b + h * p.mass_h;
    int32_t* kept = p.kept + (uint64_t)row * p.keep;
    float* mass_out = p.mass_out + (uint64_t)row * p.keep;
    for (uint32_t i = tid; i < kCopies * 257; i += THREADS) first[0][i] = 0;
    for (uint32_t i = tid; i < 4 * 256; i += THREADS) hist[0][i] = 0;
    const uint32_t len = row_length(p, b);
    const uint32_t target = min(len, p.keep);

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
    __syncthreads();
    auto key_at = [&](uint32_t j) { return held ? keys[j - begin] : key_of(mass[j], j, len, p); };

    // First digit, while the keys come in.
    constexpr int kSteps = 8;  // masses on their way at once
    for (uint32_t base = w0; base < w1; base += 32 * kSteps) {
        float m[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; u++) m[u] = base + 32 * u + lane < w1 ? mass[base + 32 * u + lane] : 0.0f;
#pragma unroll
        for (int u = 0; u < kSteps; u++) {
            const uint32_t j = base + 32 * u + lane;
            if (j >= w1) break;
            const uint32_t key = key_of(m[u], j, len, p);
            if (held) keys[j - begin] = key;
            atomicAdd(&first[lane % kCopies][key >> 24], 1u);
        }
    }
    __syncthreads();
    for (uint32_t d = tid; d < 256; d += THREADS) {
        uint32_t n = 0;
#pragma unroll
        for (uint32_t c = 0; c < kCopies; c++) n += first[c][d];
        hist[0][d] = n;
    }

    // Threshold key: its digits from the top; `want` is how many keys are still to be taken at or below the
    // decided digits.
    uint32_t prefix = 0, want = target, threshold = 0;
    uint32_t* const list = keys + cached + (w0 - begin);  // this warp's part
    uint32_t listed = 0;
#pragma unroll 1
    for (int pass = 0; pass < 4; pass++) {
        const uint32_t shift = 24 - 8 * pass;
        if (pass == 1 && held) {
            for (uint32_t base = w0; base < w1; base += 32 * kSteps) {
                uint32_t key[kSteps];
#pragma unroll
                for (int u = 0; u < kSteps; u++) key[u] = base + 32 * u + lane < w1 ? keys[base + 32 * u + lane - begin] : 0;
#pragma unroll
                for (int u = 0; u < kSteps; u++) {
                    const bool in = base + 32 * u + lane < w1 && key[u] >> 24 == prefix;
                    const uint32_t mine = __ballot_sync(0xFFFFFFFFu, in);
                    if (in) {
                        list[listed + __popc(mine & ((1u << lane) - 1))] = key[u];
                        atomicAdd(&hist[1][(key[u] >> 16) & 255], 1u);
                    }
                    listed += __popc(mine);
                }
            }
            __syncwarp();
        } else if (pass > 0) {
            for (uint32_t i = held ? lane : w0 + lane; i < (held ? listed : w1); i += 32) {
                const uint32_t key = held ? list[i] : key_of(mass[i], i, len, p);
                if ((key >> (shift + 8)) == prefix) atomicAdd(&hist[pass][(key >> shift) & 255], 1u);
            }
        }
        if (ranks > 1) {
            cluster.sync();
            if (tid < 256) {
                uint32_t n[kMaxRanks] = {}, all = 0;  // all on their way at once
#pragma unroll
                for (uint32_t r = 0; r < kMaxRanks; r++)
                    if (r < ranks) n[r] = cluster.map_shared_rank(&hist[pass][0], r)[tid];
#pragma unroll
                for (uint32_t r = 0; r < kMaxRanks; r++) all += n[r];
                hist_all[tid] = all;
            }
        }
        __syncthreads();
        if (warp == 0) {
            // Lane l holds digits 255 - 8 l down to 248 - 8 l; the threshold's is where the running count reaches `want`.
            const uint32_t* count = ranks > 1 ? hist_all : hist[pass];
            const uint4 hi = *reinterpret_cast<const uint4*>(count + 252 - 8 * lane), lo = *reinterpret_cast<const uint4*>(count + 248 - 8 * lane);
            const uint32_t mine[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
            uint32_t n = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) n += mine[i];
            uint32_t upto = n;
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= (uint32_t)o) upto += v;
            }
            uint32_t above = upto - n;
            if (above < want && want <= upto) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    if (above < want && want <= above + mine[i])
                        choice = make_uint4(255 - 8 * lane - i, above, mine[i], 0);
                    above += mine[i];
                }
            }
        }
        __syncthreads();
        const uint4 c = choice;  // digit, keys above it, keys of it
        want -= c.y;
        prefix = prefix << 8 | c.x;
        threshold = prefix << shift;
        if (c.z == want && threshold) {  // all of the bin is kept: every key from its lowest on
            threshold -= 1;
            want = 0;
            break;
        }
    }
    // Keys above the threshold are kept, and the first `want` equal to it.

    uint32_t gt = 0, eq = 0;  // of this warp's slots
#pragma unroll 4
    for (uint32_t j = w0 + lane; j < w1; j += 32) {
        const uint32_t key = key_at(j);
        gt += key > threshold;
        eq += key == threshold;
    }
    gt = __reduce_add_sync(0xFFFFFFFFu, gt);
    eq = __reduce_add_sync(0xFFFFFFFFu, eq);
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
        uint32_t sg = 0, se = 0;  // lane r: CTA r, if it is before this one
        if (lane < rank) {
            const uint2 s = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&share[0], lane));
            sg = s.x;
            se = s.y;
        }
        g += __reduce_add_sync(0xFFFFFFFFu, sg);
        e += __reduce_add_sync(0xFFFFFFFFu, se);
    }
    for (uint32_t base = w0; base < w1; base += 32 * kSteps) {
        float m[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; u++) m[u] = base + 32 * u + lane < w1 ? mass[base + 32 * u + lane] : 0.0f;
#pragma unroll
        for (int u = 0; u < kSteps; u++) {
            const uint32_t j = base + 32 * u + lane, below = (1u << lane) - 1;
            const bool in = j < w1;
            const uint32_t key = !in ? 0 : held ? keys[j - begin] : key_of(m[u], j, len, p);
            const uint32_t gs = __ballot_sync(0xFFFFFFFFu, in && key > threshold);
            uint32_t at = g + __popc(gs & below);
            bool keep = in && key > threshold;
            if (want) {  // the same for all: ties at the threshold to tell apart
                const uint32_t es = __ballot_sync(0xFFFFFFFFu, in && key == threshold);
                const uint32_t ee = e + __popc(es & below);
                keep |= in && key == threshold && ee < want;
                at += min(ee, want);
                e += __popc(es);
            }
            if (keep) {
                kept[at] = (int32_t)j;
                mass_out[at] = m[u];
            }
            g += __popc(gs);
        }
    }
    if (ranks > 1) cluster.sync();  // no CTA leaves while another reads its shared memory
}

__global__ void __launch_bounds__(kPackThreads) pack_kernel(const __grid_constant__ Params p) {
    const uint32_t row = blockIdx.y, b = row / p.cache.kv_heads, h = row % p.cache.kv_heads;
    const uint32_t total = p.keep * p.row_chunks;
    const int32_t* kept = p.kept + (uint64_t)row * p.keep;
    uzip::pdl_wait();
    // total goes up to 2^32 - 32 (host check), so an index one step further may pass 2^32
    for (uint32_t i = blockIdx.x * kPackThreads + threadIdx.x; i < total; i = next_below(i, gridDim.x * kPackThreads, total)) {
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

template <int THREADS>
int launch_select(const Params& p, uint32_t ranks, uint32_t rows, uint32_t held, cudaStream_t s) {
    static std::atomic<uint64_t> ready{0};  // a bit for each device whose limit is raised
    int dev = 0;
    UZIP_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        UZIP_CUDA_TRY(cudaFuncSetAttribute(select_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kCached * 8));
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ranks, rows);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cfg.dynamicSmemBytes = held * 8;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    UZIP_CUDA_TRY(cudaLaunchKernelEx(&cfg, select_kernel<THREADS>, p, held));
    return UZIP_OK;
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
    p.out_k = rows_of(out_k, cache->dtype, cache->sequences, cache->kv_heads, keep);
    p.out_v = rows_of(out_v, cache->dtype, cache->sequences, cache->kv_heads, keep);
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
    // A row's CTAs: as many as the SMs have room for, up to eight, while a share keeps 4096 slots.
    uint32_t ranks = 1;
    while (ranks < kMaxRanks && rows * ranks * 2 <= (uint32_t)sms && slots / ranks > 4096) ranks *= 2;
    const uint32_t per = ((slots + ranks - 1) / ranks + 31) / 32 * 32, held = per <= kCached ? per : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (per <= 4096) {  // short shares: fewer warps meet at the barriers
        if (int rc = launch_select<256>(p, ranks, rows, held, s)) return rc;
    } else {
        if (int rc = launch_select<1024>(p, ranks, rows, held, s)) return rc;
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
