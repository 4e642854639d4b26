// evict.cu -- eviction from a cache by accumulated attention weight: select
// the tokens to keep of each sequence and KV head, and pack their keys and
// values in a contiguous buffer.
//
// Select: the keep-th largest mass is found by radix selection on 32-bit keys
// whose order is the masses' (protected slots above every number, NaN below),
// eight bits a pass. Of the keys equal to the threshold the lowest slots are
// kept. One thread-block cluster takes one row (sequence, KV head), each of its
// CTAs a contiguous share of the slots; a pass's counts are summed over the
// cluster through distributed shared memory. Kept slots are written in slot
// order: each thread owns consecutive slots, so one scan of the counts gives
// every kept slot its place.
//
// Pack: bound by HBM; each kept row is read and written once, 16 bytes a lane.
#include <cooperative_groups.h>

#include <algorithm>

#include "kv_internal.cuh"

namespace cg = cooperative_groups;

namespace uzkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
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

__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ Params p) {
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ uint32_t hist[4][256];
    __shared__ uint32_t totals[256];
    __shared__ uint32_t warp_sums[2][kWarps];
    __shared__ uint32_t share[2];   // this CTA's keys above and at the threshold
    __shared__ uint32_t choice[2];  // digit, and how many keys above it
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t row = blockIdx.y, b = row / p.cache.kv_heads, h = row % p.cache.kv_heads;
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const uint32_t len = row_length(p, b);
    const uint32_t target = min(len, p.keep);
    const float* mass = p.mass + b * p.mass_b + h * p.mass_h;
    int32_t* kept = p.kept + (uint64_t)row * p.keep;
    float* mass_out = p.mass_out + (uint64_t)row * p.keep;

    if (h == 0 && rank == 0 && tid == 0) p.lengths_out[b] = (int32_t)target;
    for (uint32_t r = target + rank * kThreads + tid; r < p.keep; r += ranks * kThreads) {
        kept[r] = -1;
        mass_out[r] = 0.0f;
    }
    if (target == len) {  // keeps all (also an empty sequence)
        for (uint32_t j = rank * kThreads + tid; j < len; j += ranks * kThreads) {
            kept[j] = (int32_t)j;
            mass_out[j] = mass[j];
        }
        return;  // the whole cluster returns here
    }

    const uint32_t per = (len + ranks - 1) / ranks;
    const uint32_t begin = min(len, rank * per), end = min(len, begin + per);
    reinterpret_cast<uint32_t*>(hist)[tid] = 0;
    __syncthreads();

    // Threshold key: its digits from the top; `want` is how many keys are still to be taken below the decided digits.
    uint32_t prefix = 0, want = target;
#pragma unroll 1
    for (int pass = 0; pass < 4; pass++) {
        const uint32_t shift = 24 - 8 * pass;
        for (uint32_t j = begin + tid; j < end; j += kThreads) {
            const uint32_t key = key_of(mass[j], j, len, p);
            if (pass == 0 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[pass][(key >> shift) & 255], 1u);
        }
        cluster.sync();
        if (tid < 256) {
            uint32_t n = 0;
            for (uint32_t r = 0; r < ranks; r++) n += cluster.map_shared_rank(&hist[pass][0], r)[tid];
            totals[tid] = n;
        }
        __syncthreads();
        if (warp == 0) {
            // Lane l holds digits 255 - 8 l down to 248 - 8 l; the threshold's digit is where the running count passes want.
            uint32_t n = 0;
            for (int i = 0; i < 8; i++) n += totals[255 - 8 * lane - i];
            uint32_t upto = n;
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= (uint32_t)o) upto += v;
            }
            uint32_t above = upto - n;
            if (above < want && want <= upto) {
                for (int i = 0; i < 8; i++) {
                    const uint32_t d = 255 - 8 * lane - i;
                    if (want <= above + totals[d]) {
                        choice[0] = d;
                        choice[1] = above;
                        break;
                    }
                    above += totals[d];
                }
            }
        }
        __syncthreads();
        prefix = prefix << 8 | choice[0];
        want -= choice[1];
    }
    const uint32_t threshold = prefix;  // keys above it are kept, and the first `want` equal to it

    // Consecutive slots a thread; counts above and at the threshold, scanned over the CTA and the cluster.
    const uint32_t each = (per + kThreads - 1) / kThreads;
    const uint32_t j0 = min(end, begin + tid * each), j1 = min(end, j0 + each);
    uint32_t gt = 0, eq = 0;
    for (uint32_t j = j0; j < j1; j++) {
        const uint32_t key = key_of(mass[j], j, len, p);
        gt += key > threshold;
        eq += key == threshold;
    }
    uint32_t sg = gt, se = eq;
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t a = __shfl_up_sync(0xFFFFFFFFu, sg, o), c = __shfl_up_sync(0xFFFFFFFFu, se, o);
        if (lane >= (uint32_t)o) {
            sg += a;
            se += c;
        }
    }
    if (lane == 31) {
        warp_sums[0][warp] = sg;
        warp_sums[1][warp] = se;
    }
    __syncthreads();
    if (warp == 0) {
        uint32_t a = warp_sums[0][lane], c = warp_sums[1][lane];
        const uint32_t a0 = a, c0 = c;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, a, o), y = __shfl_up_sync(0xFFFFFFFFu, c, o);
            if (lane >= (uint32_t)o) {
                a += x;
                c += y;
            }
        }
        warp_sums[0][lane] = a - a0;
        warp_sums[1][lane] = c - c0;
        if (lane == 31) {
            share[0] = a;
            share[1] = c;
        }
    }
    cluster.sync();
    uint32_t g = warp_sums[0][warp] + sg - gt, e = warp_sums[1][warp] + se - eq;
    for (uint32_t r = 0; r < rank; r++) {
        const uint32_t* s = cluster.map_shared_rank(&share[0], r);
        g += s[0];
        e += s[1];
    }
    for (uint32_t j = j0; j < j1; j++) {
        const float m = mass[j];
        const uint32_t key = key_of(m, j, len, p);
        if (key > threshold || (key == threshold && e < want)) {
            const uint32_t at = g + min(e, want);
            kept[at] = (int32_t)j;
            mass_out[at] = m;
        }
        g += key > threshold;
        e += key == threshold;
    }
    cluster.sync();  // no CTA leaves while another reads its shared memory
}

__global__ void __launch_bounds__(kPackThreads) pack_kernel(const __grid_constant__ Params p) {
    const uint32_t row = blockIdx.y, b = row / p.cache.kv_heads, h = row % p.cache.kv_heads;
    const uint32_t total = p.keep * p.row_chunks;
    const int32_t* kept = p.kept + (uint64_t)row * p.keep;
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
    uint32_t ranks = 1;
    while (ranks < 8 && rows * ranks * 2 <= (uint32_t)sms && slots / ranks > 4096) ranks *= 2;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ranks, rows);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    UZIP_CUDA_TRY(cudaLaunchKernelEx(&cfg, select_kernel, p));
    const uint64_t chunks = (uint64_t)keep * p.row_chunks;
    const uint64_t want = std::max<uint64_t>(1, (uint64_t)sms * 32 / rows);
    const unsigned grid = (unsigned)std::min<uint64_t>((chunks + kPackThreads - 1) / kPackThreads, want);
    pack_kernel<<<dim3(grid, rows), kPackThreads, 0, s>>>(p);
    UZIP_CUDA_TRY(cudaGetLastError());
    return UZIP_OK;
}
