// kv_attend.cuh -- attention over a paged cache by warp-level matrix products:
// one pass over keys and values with the running maximum and sum of a softmax,
// the cache's tiles split over a persistent grid.
//
// Each CTA of four warps takes a run of tiles of 64 cached tokens. Keys and
// values come through a ring of shared-memory stages filled by 16-byte
// asynchronous copies that run ahead across unit boundaries; page numbers are
// looked up one step before the copies that need them. WM warps share the
// rows (16 each), 4 / WM share a tile's tokens, so that few rows still keep
// four warps busy; the token shares are merged once a unit.
#pragma once

#include <algorithm>
#include <atomic>

#include "kv_attention.cuh"

namespace uzkv {

template <typename QT, bool FP8, int DP, int WM>
struct AttCfg {
    using T = typename std::conditional<FP8, __half, QT>::type;  // type of the products
    static constexpr int kES = FP8 ? 1 : 2;
    static constexpr int kRB = DP * kES;         // bytes of a cached row in shared memory
    static constexpr int kQB = DP * 2;           // bytes of a query row
    static constexpr int kM = 16 * WM;
    static constexpr int kWN = 4 / WM;
    static constexpr int kKeys = kTile / kWN;    // tokens of a tile that a warp takes
    static constexpr int kStage = 2 * kTile * kRB;
    static constexpr int kCtas = kStage >= 65536 ? 1 : 2;  // an SM
    // Merging the token shares goes through the queries' space, which has the larger use's size.
    static constexpr int kMergeBytes = kWN > 1 ? kM * (DP + 2) * 4 : 0;
    static constexpr int kQBytes = ((kM * kQB > kMergeBytes ? kM * kQB : kMergeBytes) + 15) / 16 * 16;
    static constexpr int kFactorBytes = FP8 ? kM * 4 : 0;
    static constexpr int kOther = kQBytes + kFactorBytes + 2 * (int)kTile * 8;
    // 228 KB an SM, one of it taken by each CTA
    static constexpr int kFit = (233472 / kCtas - 1024 - kOther) / kStage;
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static_assert(kStages >= 2, "a tile in use and one on its way");
    static constexpr int kSmem = kStages * kStage + kOther;
};

template <typename QT, bool FP8, int DP, int WM>
__global__ void __launch_bounds__(kAttThreads, (AttCfg<QT, FP8, DP, WM>::kCtas)) attend_kernel(const __grid_constant__ AttParams p) {
    using C = AttCfg<QT, FP8, DP, WM>;
    using T = typename C::T;
    extern __shared__ __align__(128) char smem[];
    char* const kv = smem;
    char* const qs = smem + C::kStages * C::kStage;
    float* const factor = reinterpret_cast<float*>(qs + C::kQBytes);
    int2* const places = reinterpret_cast<int2*>(qs + C::kQBytes + C::kFactorBytes);  // [2][kTile]: page, row
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, l = lane % 4;
    const uint32_t wm = warp % WM, wn = warp / WM;
    const uint32_t D = p.cache.head_dim;

    uzip::pdl_launch_dependents();
    const uint64_t total = all_tiles(p) * p.cache.kv_heads * p.mtiles;
    const uint64_t shares = min(total, (uint64_t)p.grid);  // no share is empty
    if (blockIdx.x >= shares) return;
    const uint64_t begin = total * blockIdx.x / shares, end = total * (blockIdx.x + 1) / shares;
    const uint32_t n = (uint32_t)(end - begin);

    // Columns past the head dimension stay zero: no copy writes them.
    if (D < DP)
        for (uint32_t i = tid; i < C::kStages * C::kStage / 16; i += kAttThreads) reinterpret_cast<uint4*>(kv)[i] = make_uint4(0, 0, 0, 0);

    Unit cur = unit_at(p, begin, p.mtiles);
    Unit ahead = cur, look = cur;  // of the next tile to copy, and the next to look up
    uint32_t copied = 0, looked = 0;

    auto find = [&]() {  // place of this thread's token of the next tile to look up
        int2 at = make_int2(-1, 0);
        if (looked < n && tid < kTile) {
            const uint32_t j = look.tile * kTile + tid;
            if (j < look.span.old + look.span.fresh) {
                const Place pl = place_of(p.cache, look.b, j);
                at = make_int2(pl.page, (int)pl.row);
            }
        }
        if (looked < n) {
            looked++;
            advance(p, look, p.mtiles);
        }
        return at;
    };
    auto copy = [&]() {
        if (copied < n) {
            constexpr uint32_t kLanes = C::kRB / 16;  // a row's chunks
            const uint32_t c = tid % kLanes, live = D * C::kES / 16;
            const int2* at = places + (copied & 1) * kTile;
            char* stage = kv + (copied % C::kStages) * C::kStage;
            const char* kb = p.cache.k + ahead.h * p.cache.k_head + c * 16;
            const char* vb = p.cache.v + ahead.h * p.cache.v_head + c * 16;
            if (c < live) {
#pragma unroll
                for (uint32_t r = tid / kLanes; r < kTile; r += kAttThreads / kLanes) {
                    const int2 pl = at[r];
                    const bool ok = pl.x >= 0;
                    const uint32_t dst = smem_u32(stage) + chunk_at<C::kRB>(r, c);
                    copy16(dst, ok ? kb + pl.x * p.cache.k_page + pl.y * p.cache.k_token : p.cache.k, ok);
                    copy16(dst + kTile * C::kRB, ok ? vb + pl.x * p.cache.v_page + pl.y * p.cache.v_token : p.cache.v, ok);
                }
            }
            copied++;
            advance(p, ahead, p.mtiles);
        }
        copy_commit();
    };

    // Fill the ring: stages - 1 tiles in flight.
    if (tid < kTile) places[tid] = find(); else find();
    for (int s = 0; s < C::kStages - 1; s++) {
        const int2 next = find();
        __syncthreads();
        copy();
        if (tid < kTile) places[(copied & 1) * kTile + tid] = next;
    }

    float o[DP / 8][4], top[2], sum[2];
    bool fresh_unit = true;
    const uint32_t row0 = wm * 16 + g;  // and row0 + 8

    for (uint32_t i = 0; i < n; i++) {
        const uint64_t r0 = (uint64_t)cur.mt * C::kM;
        if (fresh_unit) {
            __syncthreads();  // the last unit's merge is done with this space
            load_queries<QT, T, DP, kAttThreads, 1>(
                p, cur.b, cur.h, (uint32_t)r0, C::kM,
                [&](uint32_t r, uint32_t c) { return reinterpret_cast<uint4*>(qs + chunk_at<C::kQB>(r, c)); }, FP8 ? factor : nullptr);
#pragma unroll
            for (int x = 0; x < DP / 8; x++)
#pragma unroll
                for (int y = 0; y < 4; y++) o[x][y] = 0.0f;
            top[0] = top[1] = -INFINITY;
            sum[0] = sum[1] = 0.0f;
        }
        const int2 next = find();
        copy_wait<C::kStages - 2>();
        __syncthreads();
        copy();
        if (tid < kTile) places[(copied & 1) * kTile + tid] = next;

        char* const stage = kv + (i % C::kStages) * C::kStage;
        const uint32_t ks = smem_u32(stage), vs = ks + kTile * C::kRB;
        const uint32_t j0 = cur.tile * kTile;
        const uint32_t mykey = wn * C::kKeys;
        float s[C::kKeys / 8][4];
#pragma unroll
        for (int x = 0; x < C::kKeys / 8; x++)
#pragma unroll
            for (int y = 0; y < 4; y++) s[x][y] = 0.0f;

        // Scores: rows by the warp's tokens.
        if (!FP8) {
#pragma unroll
            for (int kk = 0; kk < DP / 16; kk++) {
                if (kk * 16 >= D) break;
                uint32_t a[4];
                query_fragment<FP8, C::kQB>(a, qs, wm * 16, kk);
#pragma unroll
                for (int x = 0; x < C::kKeys / 16; x++) {
                    uint32_t bfr[4];
                    ldsm4(bfr, ks + chunk_at<C::kRB>(mykey + x * 16 + (lane / 16) * 8 + lane % 8, 2 * kk + (lane / 8) % 2));
                    mma16816<T>(s[2 * x], a, bfr[0], bfr[1]);
                    mma16816<T>(s[2 * x + 1], a, bfr[2], bfr[3]);
                }
            }
        } else {
#pragma unroll
            for (int kp = 0; kp < DP / 32; kp++) {
                if (kp * 32 >= D) break;
                uint32_t a[2][4];
                query_fragment<FP8, C::kQB>(a[0], qs, wm * 16, 2 * kp);
                query_fragment<FP8, C::kQB>(a[1], qs, wm * 16, 2 * kp + 1);
#pragma unroll
                for (int x = 0; x < C::kKeys / 16; x++) {
                    uint32_t r[4];
                    ldsm4(r, ks + chunk_at<C::kRB>(mykey + x * 16 + ((lane / 8) & 1) * 8 + lane % 8, 2 * kp + lane / 16));
#pragma unroll
                    for (int y = 0; y < 4; y++)
                        mma16816<T>(s[2 * x + (y & 1)], a[y >> 1], uzip::prmt(r[y], 0, 0x1404), uzip::prmt(r[y], 0, 0x3424));
                }
            }
        }

        // Running maximum and sum; scores in units of log2.
        const float f0 = FP8 ? factor[row0] : p.scale * kLog2e, f1 = FP8 ? factor[row0 + 8] : f0;
#pragma unroll
        for (int x = 0; x < C::kKeys / 8; x++) {
            s[x][0] *= f0;
            s[x][1] *= f0;
            s[x][2] *= f1;
            s[x][3] *= f1;
        }
        const bool masked = j0 + kTile > cur.span.old;
        bool dirty = false;
        uint64_t seen[2] = {~0ull, ~0ull};
        if (masked) {
            // A value that a row does not see must not reach it through 0 * NaN: non-finite values of new tokens
            // leave the tile here and are added below to the rows that see them.
            int found = 0;
            for (uint32_t c = tid; c < kTile * (C::kRB / 16); c += kAttThreads) {
                const uint32_t r = c / (C::kRB / 16);
                if (j0 + r < cur.span.old) continue;
                uint32_t* w = reinterpret_cast<uint32_t*>(stage + kTile * C::kRB + chunk_at<C::kRB>(r, c % (C::kRB / 16)));
#pragma unroll
                for (int y = 0; y < 4; y++) {
                    uint32_t v = w[y], keep = 0;
                    if (FP8) {
                        for (int z = 0; z < 4; z++) keep |= ((v >> (8 * z)) & 0x7C) != 0x7C ? 0xFFu << (8 * z) : 0;
                    } else {
                        constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
                        for (int z = 0; z < 2; z++) keep |= ((v >> (16 * z)) & kExp) != kExp ? 0xFFFFu << (16 * z) : 0;
                    }
                    if (keep != 0xFFFFFFFFu) {
                        w[y] = v & keep;
                        found = 1;
                    }
                }
            }
            dirty = __syncthreads_or(found);
            seen[0] = seen_bits(p, cur.b, cur.span, (uint32_t)r0 + row0, j0) >> mykey;
            seen[1] = seen_bits(p, cur.b, cur.span, (uint32_t)r0 + row0 + 8, j0) >> mykey;
#pragma unroll
            for (int x = 0; x < C::kKeys / 8; x++)
#pragma unroll
                for (int y = 0; y < 4; y++)
                    if (!((seen[y >> 1] >> (x * 8 + 2 * l + (y & 1))) & 1)) s[x][y] = -INFINITY;
        }
        float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < C::kKeys / 8; x++) {
            most[0] = fmaxf(most[0], fmaxf(s[x][0], s[x][1]));
            most[1] = fmaxf(most[1], fmaxf(s[x][2], s[x][3]));
        }
        float ref[2], fade[2];
        bool moved = false;
#pragma unroll
        for (int y = 0; y < 2; y++) {
            most[y] = fmaxf(most[y], __shfl_xor_sync(0xFFFFFFFFu, most[y], 1));
            most[y] = fmaxf(most[y], __shfl_xor_sync(0xFFFFFFFFu, most[y], 2));
            const float now = fmaxf(top[y], most[y]);
            fade[y] = top[y] == -INFINITY ? 0.0f : exp2_fast(top[y] - now);  // 0: nothing so far
            moved |= now != top[y];
            top[y] = now;
            ref[y] = now == -INFINITY ? 0.0f : now - kLift<T>;
        }
        if (__any_sync(0xFFFFFFFFu, moved)) {
            sum[0] *= fade[0];
            sum[1] *= fade[1];
#pragma unroll
            for (int x = 0; x < DP / 8; x++) {
                o[x][0] *= fade[0];
                o[x][1] *= fade[0];
                o[x][2] *= fade[1];
                o[x][3] *= fade[1];
            }
        }
        uint32_t pr[C::kKeys / 8][2];  // weights, rounded to the products' type; their sum is of the unrounded ones
#pragma unroll
        for (int x = 0; x < C::kKeys / 8; x++) {
            const float e0 = exp2_fast(s[x][0] - ref[0]), e1 = exp2_fast(s[x][1] - ref[0]);
            const float e2 = exp2_fast(s[x][2] - ref[1]), e3 = exp2_fast(s[x][3] - ref[1]);
            sum[0] += e0 + e1;
            sum[1] += e2 + e3;
            pr[x][0] = pack2<T>(e0, e1);
            pr[x][1] = pack2<T>(e2, e3);
        }

        // Values.
#pragma unroll
        for (int ksx = 0; ksx < C::kKeys / 16; ksx++) {
            const uint32_t a[4] = {pr[2 * ksx][0], pr[2 * ksx][1], pr[2 * ksx + 1][0], pr[2 * ksx + 1][1]};
            const uint32_t key = mykey + ksx * 16 + ((lane / 8) & 1) * 8 + lane % 8;
            if (!FP8) {
#pragma unroll
                for (int x = 0; x < DP / 16; x++) {
                    if (x * 16 >= D) break;
                    uint32_t bfr[4];
                    ldsm4_t(bfr, vs + chunk_at<C::kRB>(key, 2 * x + lane / 16));
                    mma16816<T>(o[2 * x], a, bfr[0], bfr[1]);
                    mma16816<T>(o[2 * x + 1], a, bfr[2], bfr[3]);
                }
            } else {
#pragma unroll
                for (int x = 0; x < DP / 32; x++) {
                    if (x * 32 >= D) break;
                    uint32_t r[4];
                    ldsm4_t(r, vs + chunk_at<C::kRB>(key, 2 * x + lane / 16));
#pragma unroll
                    for (int y = 0; y < 2; y++) {  // 16 columns: the even ones, then the odd ones
                        mma16816<T>(o[4 * x + 2 * y], a, uzip::prmt(r[2 * y], 0, 0x2404), uzip::prmt(r[2 * y + 1], 0, 0x2404));
                        mma16816<T>(o[4 * x + 2 * y + 1], a, uzip::prmt(r[2 * y], 0, 0x3414), uzip::prmt(r[2 * y + 1], 0, 0x3414));
                    }
                }
            }
        }
        // Column of o[x][y] (and y + 2): x * 8 + 2 l + y, or with the even and odd columns apart.
        auto column = [&](int x, int y) { return FP8 ? (x / 2) * 16 + 4 * l + 2 * y + (x & 1) : x * 8 + 2 * l + y; };

        if (dirty) {
            const uint32_t upto = cur.span.old + cur.span.fresh;
            for (uint32_t k = 0; k < C::kKeys; k++) {
                const uint32_t j = j0 + mykey + k;
                if (j < cur.span.old || j >= upto) continue;
                const Place pl = place_of(p.cache, cur.b, j);
                if (pl.page < 0) continue;
                const char* v = v_row(p.cache, pl, cur.h);
#pragma unroll
                for (int x = 0; x < DP / 8; x++)
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        const uint32_t d = column(x, y);
                        if (d >= D) continue;
                        const float e = FP8 ? to_f32(reinterpret_cast<const E5M2*>(v)[d]) : to_f32(reinterpret_cast<const T*>(v)[d]);
                        if (isfinite(e)) continue;
                        if ((seen[0] >> k) & 1) o[x][y] += e;
                        if ((seen[1] >> k) & 1) o[x][y + 2] += e;
                    }
            }
        }

        // End of the unit or of this CTA's run: a whole unit's rows are done, a part goes to the workspace.
        const Unit done = cur;
        const bool to_end = done.tile + 1 == done.tiles;
        advance(p, cur, p.mtiles);
        static_assert(kTile == 64, "seen_bits");
        if (!to_end && i + 1 < n) {
            fresh_unit = false;
            continue;
        }
        fresh_unit = true;
        for (int y = 0; y < 2; y++) {
            sum[y] += __shfl_xor_sync(0xFFFFFFFFu, sum[y], 1);
            sum[y] += __shfl_xor_sync(0xFFFFFFFFu, sum[y], 2);
        }
        float mref[2] = {top[0] == -INFINITY ? 0.0f : top[0] - kLift<T>, top[1] == -INFINITY ? 0.0f : top[1] - kLift<T>};
        if (C::kWN > 1) {
            // Token shares, one warp after the other, through the queries' space.
            float* box = reinterpret_cast<float*>(qs);
            float* stat = box + C::kM * DP;
            for (int w = C::kWN - 1; w >= 0; w--) {
                __syncthreads();
                if ((int)wn != w) continue;
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    const uint32_t r = row0 + 8 * y;
                    float mine = 1.0f, theirs = 0.0f;
                    if (w < C::kWN - 1) {
                        const float om = stat[2 * r], os = stat[2 * r + 1];
                        const float both = sum[y] == 0.0f ? om : os == 0.0f ? mref[y] : fmaxf(om, mref[y]);
                        mine = sum[y] == 0.0f ? 0.0f : exp2_fast(mref[y] - both);
                        theirs = os == 0.0f ? 0.0f : exp2_fast(om - both);
                        sum[y] = sum[y] * mine + os * theirs;
                        mref[y] = both;
                    }
#pragma unroll
                    for (int x = 0; x < DP / 8; x++) {
                        float2* at = reinterpret_cast<float2*>(box + r * DP + (x ^ (r & 7)) * 8 + 2 * l);  // rows apart in the banks
                        float a0 = o[x][2 * y], a1 = o[x][2 * y + 1];
                        if (w < C::kWN - 1) {
                            const float2 v = *at;
                            a0 = a0 * mine + v.x * theirs;
                            a1 = a1 * mine + v.y * theirs;
                            o[x][2 * y] = a0;
                            o[x][2 * y + 1] = a1;
                        }
                        if (w) *at = make_float2(a0, a1);
                    }
                    __syncwarp();
                    if (w && l == 0) {
                        stat[2 * r] = mref[y];
                        stat[2 * r + 1] = sum[y];
                    }
                }
            }
        }
        if (wn != 0) continue;
        const bool started = done.tile <= i;  // its first tile is in this run
        if (started && to_end) {
#pragma unroll
            for (int y = 0; y < 2; y++) {
                const uint32_t row = (uint32_t)r0 + row0 + 8 * y;
                if (row >= p.rows) continue;
                const uint32_t t = row / p.group, hq = done.h * p.group + row % p.group;
                const bool none = t >= done.span.fresh || sum[y] == 0.0f;
                const float inv = none ? 0.0f : 1.0f / sum[y];
                char* out = p.out.p + done.b * p.out.b + t * p.out.t + (uint64_t)hq * p.out.h;
                if (!FP8) {
#pragma unroll
                    for (int x = 0; x < DP / 8; x++)
                        if ((uint32_t)x * 8 < D)
                            *reinterpret_cast<uint32_t*>(out + 2 * (x * 8 + 2 * l)) =
                                none ? 0u : pack2<QT>(o[x][2 * y] * inv, o[x][2 * y + 1] * inv);
                } else {
#pragma unroll
                    for (int x = 0; x < DP / 16; x++)
                        if ((uint32_t)x * 16 < D)
                            *reinterpret_cast<uint2*>(out + 2 * (x * 16 + 4 * l)) =
                                none ? make_uint2(0, 0)
                                     : make_uint2(pack2<QT>(o[2 * x][2 * y] * inv, o[2 * x + 1][2 * y] * inv),
                                                  pack2<QT>(o[2 * x][2 * y + 1] * inv, o[2 * x + 1][2 * y + 1] * inv));
                }
                if (p.lse && l == 0)
                    p.lse[((uint64_t)done.b * p.tokens + t) * p.q_heads + hq] = none ? -INFINITY : (mref[y] + log2f(sum[y])) * kLn2;
            }
        } else {
            float* part = p.partial + ((uint64_t)blockIdx.x * 2 + (started ? 1 : 0)) * partial_floats(p);
#pragma unroll
            for (int y = 0; y < 2; y++) {
                const uint32_t r = row0 + 8 * y, row = (uint32_t)r0 + r;
                if (row >= p.rows) continue;
#pragma unroll
                for (int x = 0; x < DP / 8; x++) {
                    if (column(x, 0) >= D) continue;
                    if (!FP8) {
                        *reinterpret_cast<float2*>(part + (uint64_t)r * DP + column(x, 0)) = make_float2(o[x][2 * y], o[x][2 * y + 1]);
                    } else if (x % 2 == 0) {
                        *reinterpret_cast<float4*>(part + (uint64_t)r * DP + column(x, 0)) =
                            make_float4(o[x][2 * y], o[x + 1][2 * y], o[x][2 * y + 1], o[x + 1][2 * y + 1]);
                    }
                }
                if (l == 0) {
                    part[(uint64_t)C::kM * DP + 2 * r] = mref[y];
                    part[(uint64_t)C::kM * DP + 2 * r + 1] = row / p.group < done.span.fresh ? sum[y] : 0.0f;
                }
            }
        }
    }
}

template <typename QT, bool FP8, int DP, int WM>
int launch_attend_as(AttParams& p, int sms, cudaStream_t stream) {
    using C = AttCfg<QT, FP8, DP, WM>;
    static std::atomic<uint64_t> ready{0};  // a bit for each device whose limit is raised
    int dev = 0;
    UZIP_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        UZIP_CUDA_TRY(cudaFuncSetAttribute(attend_kernel<QT, FP8, DP, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    p.m = C::kM;
    p.mtiles = (p.rows + C::kM - 1) / C::kM;
    p.dp = DP;
    p.shift = 6;
    static_assert(kTile == 1u << 6, "tile");
    p.grid = std::min<uint32_t>((uint32_t)sms * C::kCtas, kMaxAttGrid);
    attend_kernel<QT, FP8, DP, WM><<<p.grid, kAttThreads, C::kSmem, stream>>>(p);
    UZIP_CUDA_TRY(cudaGetLastError());
    return UZIP_OK;
}

// Rows a CTA takes at once: the fewest that hold all, up to 64.
template <typename QT, bool FP8, int DP>
int launch_attend_rows(AttParams& p, int sms, cudaStream_t s) {
    if (p.rows <= 16) return launch_attend_as<QT, FP8, DP, 1>(p, sms, s);
    if (p.rows <= 32) return launch_attend_as<QT, FP8, DP, 2>(p, sms, s);
    return launch_attend_as<QT, FP8, DP, 4>(p, sms, s);
}

template <typename QT, bool FP8>
int launch_attend(AttParams& p, int sms, cudaStream_t s) {
    if (p.cache.head_dim <= 64) return launch_attend_rows<QT, FP8, 64>(p, sms, s);
    if (p.cache.head_dim <= 128) return launch_attend_rows<QT, FP8, 128>(p, sms, s);
    return launch_attend_rows<QT, FP8, 256>(p, sms, s);
}

}  // namespace uzkv
