// kv_mass.cuh -- the attention weight that each cached token collects, on the
// tensor cores.
//
// With the rows' log-sum-exp given, a weight is exp2(s * f - e) with e of the
// row alone, and a token's mass their sum over rows: no running maximum, no
// second product. The product is taken with the cached tokens along M:
// S^T = K Q^T, 128 tokens by up to 256 rows, so that in tensor memory a lane
// is a token and the sum over rows stays within a thread, in one fixed order.
// Any number of rows costs only its own columns (a multiple of 16).
//
// Bound: HBM for few rows, else the sums: an exponential a row and token (32 a clock on an SM) and what surrounds it.
// Measured: 256 rows of 128 over 131,072 tokens of 8 heads: 90 us (floor 41 by bytes, 36 by products); 20 rows of 64 over 24
// E5M2 sequences of up to 3,001 tokens: 23 us, most of it startup and the units' ends.
//
// One CTA an SM takes a run of tiles (kv_attention.cuh's split). Its warps: 13
// brings keys to a ring of operand tiles by bulk copies; 0-3 load the rows'
// queries and factors once a unit, widen E5M2 keys, which land as bytes, to
// FP16 tiles, and do the copies where pages do not allow bulk ones; 12 issues
// the products into two buffers of tensor memory; 4-7 and 8-11 take turns at
// the tiles, sum, add the decayed old mass and store. More than 256 rows (128 for heads above 128) go in chunks: the
// CTA passes over its tiles of the unit once a chunk, adding to what the same
// thread stored before.
#pragma once

#include <algorithm>
#include <atomic>

#include "kv_tcgen05.cuh"

namespace uzkv {

constexpr int kMassThreads = 14 * 32;
constexpr uint32_t kMassTile = 128;

template <typename QT, bool FP8, int DP>
struct MassCfg {
    using T = typename std::conditional<FP8, __half, QT>::type;
    static constexpr uint32_t kMaxN = DP <= 128 ? 256 : 128;          // rows of a chunk
    static constexpr uint32_t kQBytes = kMaxN * DP * 2;               // one chunk's queries, or two smaller ones'
    static constexpr uint32_t kTileBytes = kMassTile * DP * 2;
    static constexpr uint32_t kRawBytes = kMassTile * DP;             // E5M2 bytes of a tile
    static constexpr uint32_t kRoom = 227 * 1024 - 8192;              // less factors and barriers
    // 16-bit keys: as many operand tiles as fit. E5M2: few operand tiles, the rest of the space for bytes on their way.
    static constexpr uint32_t kFit = (kRoom - kQBytes) / kTileBytes;
    static constexpr uint32_t kTiles = FP8 ? (DP <= 128 ? 2 : 1) : (kFit > 8 ? 8 : kFit);
    static constexpr uint32_t kRaw = FP8 ? (DP <= 128 ? 4 : 2) : 0;
    static constexpr uint32_t kRing = FP8 ? kRaw : kTiles;            // tiles on their way
    static constexpr uint32_t kSmem = kQBytes + kTiles * kTileBytes + kRaw * kRawBytes + 8192;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kTiles >= 1, "operand tiles");
};

// The runs of tiles of one unit and chunk that a CTA passes over; all roles walk the same list.
struct MassWalk {
    Unit u;
    uint64_t end;
    uint32_t chunk, count, units;
    __device__ __forceinline__ MassWalk(const Unit& first, uint64_t e) : u(first), end(e), chunk(0), units(0) { take(); }
    __device__ __forceinline__ void take() { count = valid() ? (uint32_t)min((uint64_t)(u.tiles - u.tile), end - u.pos) : 0; }
    __device__ __forceinline__ bool valid() const { return u.pos < end; }
    __device__ __forceinline__ void next(const AttParams& p) {
        if (++chunk < p.mtiles) return;
        chunk = 0;
        u.tile += count - 1;
        u.pos += count - 1;
        advance(p, u, 1);
        units++;
        take();
    }
    // Which of the two accumulators and summing groups takes tile i: turns over tiles and units, the same in every
    // chunk, so that the thread that adds a later chunk to a token's mass is the one that stored it.
    __device__ __forceinline__ uint32_t turn(uint32_t i) const { return (i + units) & 1; }
};

template <typename QT, bool FP8, int DP, bool TMA>
__global__ void __launch_bounds__(kMassThreads, 1) mass_kernel(const __grid_constant__ AttParams p, const __grid_constant__ Maps maps) {
    using C = MassCfg<QT, FP8, DP>;
    using T = typename C::T;
    extern __shared__ __align__(1024) char smem[];
    char* const qs = smem;
    char* const tiles = qs + C::kQBytes;
    char* const raws = tiles + C::kTiles * C::kTileBytes;
    float* const rowf = reinterpret_cast<float*>(raws + C::kRaw * C::kRawBytes);  // [2][2][256]: factors; exponents, negative
    uint64_t* const bars = reinterpret_cast<uint64_t*>(rowf + 1024);
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(bars + 40);
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const uint32_t D = p.cache.head_dim, N = p.m;
    const uint32_t qbuf = 2 * N * DP * 2 <= C::kQBytes ? 2 : 1;  // queries of two units at once where they fit
    const uint32_t full = smem_u32(bars), freed = full + 8 * 8, q_full = full + 16 * 8, q_freed = full + 18 * 8,
                   s_full = full + 20 * 8, s_freed = full + 22 * 8, landed = full + 24 * 8, raw_freed = full + 32 * 8;
    uint32_t columns = 32;
    while (columns < 2 * N) columns *= 2;

    if (tid == 0) {
        for (uint32_t i = 0; i < 8; i++) {
            bar_init(full + 8 * i, TMA && !FP8 ? 1 : 4);  // the bulk copies, or the four warps that bring or widen
            bar_init(freed + 8 * i, 1);                   // the products' commit
            bar_init(landed + 8 * i, 1);                  // E5M2 bytes: the bulk copies
            bar_init(raw_freed + 8 * i, 4);               // ... and the four warps that widen
        }
        for (uint32_t i = 0; i < 2; i++) {
            bar_init(q_full + 8 * i, 4);
            bar_init(q_freed + 8 * i, 9);  // the products' commit and the eight summing warps
            bar_init(s_full + 8 * i, 1);
            bar_init(s_freed + 8 * i, 4);  // the four warps of the buffer's group
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) tc_alloc(smem_u32(tmem_at), columns);
    if (D < DP && (FP8 || !TMA)) {  // columns past the head dimension stay zero: no copy writes them
        for (uint32_t i = tid; i < C::kTiles * C::kTileBytes / 16; i += kMassThreads) reinterpret_cast<uint4*>(tiles)[i] = make_uint4(0, 0, 0, 0);
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;

    const Split split = split_of(p);
    const Run run = run_of(p, split, 1);
    Unit first{};
    first.pos = ~0ull;
    if (run.begin != run.end) first = unit_at(p, split, run.begin, 1);
    bool ok = true;

    if (warp < 4) {
        // ---- copies
        constexpr uint32_t kES = FP8 ? 1 : 2, kLanes = DP * kES / 16;  // a row's chunks
        constexpr uint32_t kRing = C::kRing;
        const uint32_t c = lane % kLanes, live = D * kES / 16;
        MassWalk cw(first, run.end);  // of the next tile to copy
        uint32_t cs = 0, copied = 0;  // its place in the run, and how many are copied
        Place ahead{0, 0};
        bool used = false;  // whether the next tile has a token for this lane
        auto find = [&]() {
            const uint32_t j = (cw.u.tile + cs) * kMassTile + warp * 32 + lane;
            used = cw.valid() && j < cw.u.span.old + cw.u.span.fresh;
            if (used) ahead = look_up(p.cache, cw.u.b, j);
        };
        if (!TMA) find();
        auto copy = [&]() {
            if (TMA) return;
            if (ok && cw.valid()) {
                // A warp takes 32 of the tile's rows: each lane finds one, then the warp copies them row by row.
                if (!FP8 && copied >= kRing) ok = warp_wait(freed + 8 * (copied % kRing), (copied / kRing - 1) & 1);
                if (FP8) __syncwarp();  // this warp has widened what the slot held: it copies only its own rows
                const Place now = used ? checked(p.cache, ahead) : Place{-1, 0};
                const char* row = now.page >= 0 ? k_row(p.cache, now, cw.u.h) : nullptr;
                char* slot = (FP8 ? raws : tiles) + (copied % kRing) * (FP8 ? C::kRawBytes : C::kTileBytes);
#pragma unroll 8
                for (uint32_t i = 0; i < kLanes; i++) {
                    const uint32_t r = i * (32 / kLanes) + lane / kLanes;
                    const char* src = reinterpret_cast<const char*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(row), r));
                    const uint32_t R = warp * 32 + r;
                    const uint32_t at = FP8 ? row_chunk<DP>(kMassTile, R, c) : swizzled(kMassTile, R, c);
                    if (c < live) copy16(smem_u32(slot) + at, src ? src + c * 16 : p.cache.k, src != nullptr);
                }
                copied++;
                if (++cs == cw.count) {
                    cs = 0;
                    cw.next(p);
                }
                find();
            }
            copy_commit();
        };
        uint32_t seg = 0, sent = 0;
        for (uint32_t i = 0; i < kRing - 1; i++) copy();
        for (MassWalk w(first, run.end); w.valid() && ok; w.next(p), seg++) {
            // The rows' queries, factors and exponents.
            const uint32_t qb = seg % qbuf, fb = seg % 2;
            if (seg >= qbuf) ok = warp_wait(q_freed + 8 * qb, (seg / qbuf - 1) & 1);
            if (!ok) break;
            const uint32_t row0 = w.chunk * N;
            char* q = qs + qb * N * DP * 2;
            float* f = rowf + fb * 512;
            load_queries<QT, T, DP, 128>(
                p, tid, w.u.b, w.u.h, row0, N, [&](uint32_t r, uint32_t ch) { return reinterpret_cast<uint4*>(q + swizzled(N, r, ch)); },
                f);
            for (uint32_t r = tid; r < N; r += 128) {
                const uint32_t row = row0 + r, t = row / p.group;
                float e = -INFINITY;  // a row that adds nothing
                if (row < p.rows && t < w.u.span.fresh) {
                    const float lse = p.lse[((uint64_t)w.u.b * p.tokens + t) * p.q_heads + w.u.h * p.group + row % p.group];
                    const float wt = p.weights ? p.weights[(uint64_t)w.u.b * p.tokens + t] : 1.0f;
                    if (lse != -INFINITY && wt != 0.0f) e = p.weights ? log2f(wt) - lse * kLog2e : -lse * kLog2e;
                }
                f[256 + r] = e;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(q_full + 8 * (seg % 2));
            for (uint32_t i = 0; i < w.count && ok && (FP8 || !TMA); i++, sent++) {
                if (TMA) ok = warp_wait(landed + 8 * (sent % C::kRing), (sent / C::kRing) & 1);
                else copy_wait<kRing - 2>();
                if (!ok) break;
                if (FP8) {
                    // Widen this warp's rows of the tile: 16 bytes to two chunks of eight FP16.
                    if (sent >= C::kTiles) ok = warp_wait(freed + 8 * (sent % C::kTiles), (sent / C::kTiles - 1) & 1);
                    __syncwarp();
                    const char* raw = raws + (sent % kRing) * C::kRawBytes;
                    char* tile = tiles + (sent % C::kTiles) * C::kTileBytes;
                    constexpr uint32_t kBatch = kLanes < 8 ? kLanes : 8;  // all read before the first is written
                    if (c < live)
#pragma unroll
                        for (uint32_t x0 = 0; x0 < kLanes; x0 += kBatch) {
                            uint4 v[kBatch];
#pragma unroll
                            for (uint32_t x = 0; x < kBatch; x++)
                                v[x] = *reinterpret_cast<const uint4*>(raw + row_chunk<DP>(kMassTile, warp * 32 + (x0 + x) * (32 / kLanes) + lane / kLanes, c));
#pragma unroll
                            for (uint32_t x = 0; x < kBatch; x++) {
                                const uint32_t R = warp * 32 + (x0 + x) * (32 / kLanes) + lane / kLanes;
                                *reinterpret_cast<uint4*>(tile + swizzled(kMassTile, R, 2 * c)) = widen(v[x].x, v[x].y);
                                *reinterpret_cast<uint4*>(tile + swizzled(kMassTile, R, 2 * c + 1)) = widen(v[x].z, v[x].w);
                            }
                        }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(full + 8 * (sent % C::kTiles));
                    if (TMA) bar_arrive(raw_freed + 8 * (sent % C::kRing));
                }
                copy();
            }
        }
        if (!TMA) copy_wait<0>();
    } else if (warp == 13) {
        // ---- bulk copies
        if (TMA) {
            using Feed = TmaFeed<kMassTile, FP8 ? DP : DP * 2>;
            char* const ring = FP8 ? raws : tiles;
            const uint32_t done = FP8 ? landed : full, again = FP8 ? raw_freed : freed;
            MassWalk w(first, run.end);
            Unit u = first;
            Feed feed;
            feed.find(p, maps, u, w.valid());
            uint32_t i = 0, at = 0;  // tile of the run, and of its unit's part
            while (w.valid() && ok) {
                const Feed now = feed;
                const uint32_t h = u.h, s = i % C::kRing;
                if (++at == w.count) {
                    at = 0;
                    w.next(p);
                    u = w.u;
                } else {
                    u.tile++;
                }
                feed.find(p, maps, u, w.valid());
                if (i >= C::kRing) ok = warp_wait(again + 8 * s, (i / C::kRing - 1) & 1);
                if (!ok) break;
                if (lane == 0) bar_expect(done + 8 * s, now.bytes(maps));
                __syncwarp();
                now.copy(p, maps, &maps.k, h, smem_u32(ring + s * (FP8 ? C::kRawBytes : C::kTileBytes)), done + 8 * s);
                i++;
            }
            for (uint32_t k = i > C::kRing ? i - C::kRing : 0; k < i; k++)  // no copy outlives the CTA
                ok &= warp_wait(done + 8 * (k % C::kRing), (k / C::kRing) & 1);
        }
    } else if (warp == 12) {
        // ---- products, by one lane
        if (lane == 0) {
            const uint32_t idesc = mma_desc<T>(kMassTile, N), q_block = N * 128 >> 4;
            const uint64_t tiles_desc = tile_desc(smem_u32(tiles));
            uint32_t seg = 0, k = 0, uses[2] = {0, 0};
            for (MassWalk w(first, run.end); w.valid() && ok; w.next(p), seg++) {
                ok = bar_wait(q_full + 8 * (seg % 2), (seg / 2) & 1);
                const uint64_t q_desc = tile_desc(smem_u32(qs) + seg % qbuf * N * DP * 2);  // offsets add to its low bits
                for (uint32_t i = 0; i < w.count && ok; i++, k++) {
                    const uint32_t s = k % C::kTiles, side = w.turn(i), used = side ? uses[1]++ : uses[0]++;
                    ok = bar_wait(full + 8 * s, (k / C::kTiles) & 1);
                    if (ok && used) ok = bar_wait(s_freed + 8 * side, (used - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a = tiles_desc + s * (C::kTileBytes >> 4);
                    if (D > DP * 3 / 4) tc_mma_steps<DP / 16>(tmem + side * N, a, kMassTile * 128 >> 4, q_desc, q_block, idesc);
                    else tc_mma_steps<DP * 3 / 64>(tmem + side * N, a, kMassTile * 128 >> 4, q_desc, q_block, idesc);
                    tc_commit(freed + 8 * s);
                    tc_commit(s_full + 8 * side);
                }
                if (ok) tc_commit(q_freed + 8 * (seg % qbuf));
            }
        }
        __syncwarp();
    } else {
        // ---- sums: a thread is a cached token
        const uint32_t group = warp < 8 ? 0 : 1, quarter = warp % 4;
        uint32_t seg = 0, used = 0;
        for (MassWalk w(first, run.end); w.valid() && ok; w.next(p), seg++) {
            const Span sp = w.u.span;
            const float *f = rowf + seg % 2 * 512, *e = f + 256;
            const int64_t row_at = w.u.b * p.mass_b + w.u.h * p.mass_h;
            ok = warp_wait(q_full + 8 * (seg % 2), (seg / 2) & 1);
            for (uint32_t i = 0; i < w.count && ok; i++) {
                if (w.turn(i) != group) continue;
                const uint32_t j0 = (w.u.tile + i) * kMassTile, j = j0 + quarter * 32 + lane;
                // What the sum is added to: on its way meanwhile.
                const bool decayed = w.chunk == 0;
                float before = 0.0f;
                if (j < p.slots && !decayed) before = p.mass_out[row_at + j];
                else if (j < p.slots && p.mass_in && j < sp.old) before = p.mass_in[row_at + j];
                ok = warp_wait(s_full + 8 * group, used++ & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = tmem + group * N + (quarter * 32 << 16);
                float acc = 0.0f;
                bool guard = j0 + quarter * 32 + 32 > sp.old;
                if (!guard) {
                    // 32 columns at a time, the next ones on their way meanwhile.
                    uint32_t v[2][32];
                    uint64_t part[4] = {0, 0, 0, 0};
                    const uint64_t f1 = pair(fabsf(p.scale) * kLog2e, fabsf(p.scale) * kLog2e);
                    auto columns = [&](const uint32_t* x, uint32_t c0, auto count) {
#pragma unroll
                        for (int i = 0; i < decltype(count)::value; i += 4) {
                            const ulonglong2 en = *reinterpret_cast<const ulonglong2*>(e + c0 + i);
                            ulonglong2 fn = make_ulonglong2(f1, f1);
                            if (FP8) fn = *reinterpret_cast<const ulonglong2*>(f + c0 + i);  // rows have their own powers of two
                            const float2 a = unpair(fma2(pair(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), fn.x, en.x));
                            const float2 b = unpair(fma2(pair(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), fn.y, en.y));
                            part[i / 2 % 4] = add2(part[i / 2 % 4], pair(exp2_fast(a.x), exp2_fast(a.y)));
                            part[i / 2 % 4 + 1] = add2(part[i / 2 % 4 + 1], pair(exp2_fast(b.x), exp2_fast(b.y)));
                        }
                    };
                    const uint32_t whole = N / 32 * 32;
                    if (whole) tc_ld32(v[0], at);
                    for (uint32_t c0 = 0; c0 < whole; c0 += 64) {
                        tc_wait_ld();
                        if (c0 + 32 < whole) tc_ld32(v[1], at + c0 + 32);
                        columns(v[0], c0, std::integral_constant<int, 32>{});
                        if (c0 + 32 < whole) {
                            tc_wait_ld();
                            if (c0 + 64 < whole) tc_ld32(v[0], at + c0 + 64);
                            columns(v[1], c0 + 32, std::integral_constant<int, 32>{});
                        }
                    }
                    if (whole < N) {
                        tc_ld16(reinterpret_cast<float*>(v[0]), at + whole);
                        tc_wait_ld();
                        columns(v[0], whole, std::integral_constant<int, 16>{});
                    }
                    part[0] = add2(part[0], part[2]);
                    part[1] = add2(part[1], part[3]);
                    const float2 sum = unpair(add2(part[0], part[1]));
                    acc = sum.x + sum.y;
                    // A key that is not finite makes NaN of rows that add nothing too: take those rows out.
                    guard = __any_sync(0xFFFFFFFFu, acc != acc);
                }
                if (guard) {
                    // Which new tokens see this lane's: 32 tokens' bits at a time, for the rows that are theirs.
                    acc = 0.0f;
                    const uint32_t row0 = w.chunk * N, u = j - sp.old;
                    uint32_t t = row0 / p.group, left = p.group - row0 % p.group;  // rows left of token t
                    const bool in = j < sp.old + sp.fresh, old = j < sp.old;
                    const int64_t* words = p.mask && in && !old ? p.mask + w.u.b * p.mask_b + (u >> 6) : nullptr;
                    auto bits_from = [&](uint32_t first) {
                        uint32_t bits = !in ? 0 : old ? 0xFFFFFFFFu : 0;
                        if (in && !old)
#pragma unroll 8
                            for (uint32_t i = 0; i < 32; i++) {
                                const uint32_t tok = first + i;
                                if (tok < sp.fresh && (p.mask ? (bool)(words[(uint64_t)tok * p.mask_words] >> (u & 63) & 1) : u <= tok)) bits |= 1u << i;
                            }
                        return bits;
                    };
                    uint32_t first_bit = t, bits = bits_from(t);
                    for (uint32_t c0 = 0; c0 < N; c0 += 16) {
                        float v[16];
                        tc_ld16(v, at + c0);
                        uint32_t see = 0;  // of these 16 rows, a token's at once
                        for (uint32_t x = 0; x < 16;) {
                            const uint32_t n = min(left, 16 - x);
                            see |= (bits & 1) ? ((1u << n) - 1) << x : 0;
                            x += n;
                            left -= n;
                            if (left == 0) {  // the same for all lanes
                                left = p.group;
                                bits >>= 1;
                                if (++t == first_bit + 32) {
                                    first_bit = t;
                                    bits = bits_from(t);
                                }
                            }
                        }
                        tc_wait_ld();
#pragma unroll
                        for (int x = 0; x < 16; x++) {
                            const float en = e[c0 + x], m = exp2_fast(v[x] * f[c0 + x] + en);
                            acc += (see >> x & 1) && en != -INFINITY ? m : 0.0f;
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(s_freed + 8 * group);
                if (j < p.slots) p.mass_out[row_at + j] = acc + (decayed ? p.decay * before : before);
            }
            // This warp's last read of the unit's factors is behind it.
            __syncwarp();
            if (lane == 0 && ok) bar_arrive(q_freed + 8 * (seg % qbuf));
        }
        // Slots that no tile covers: past the new tokens, or all of a sequence that has none.
        const uint32_t rows = p.cache.sequences * p.cache.kv_heads;
        for (uint32_t r = blockIdx.x; r < rows; r += gridDim.x) {
            const uint32_t b = r / p.cache.kv_heads, h = r % p.cache.kv_heads;
            const Span sp = span_of(p.cache, p.counts, p.tokens, b);
            const int64_t row_at = b * p.mass_b + h * p.mass_h;
            for (uint64_t j = (uint64_t)tiles_of(p, sp) * kMassTile + (tid - 128); j < p.slots; j += 256)
                p.mass_out[row_at + j] = p.mass_in && j < sp.old ? p.decay * p.mass_in[row_at + j] : 0.0f;
        }
    }
    if (!ok && p.cache.status) *p.cache.status = UZIP_ERR_TIMEOUT;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tc_free(tmem, columns);
}

template <typename QT, bool FP8, int DP, bool TMA>
int launch_mass_by(AttParams& p, const Maps& maps, cudaStream_t stream) {
    using C = MassCfg<QT, FP8, DP>;
    static std::atomic<uint64_t> ready{0};  // a bit for each device whose limit is raised
    int dev = 0;
    UZIP_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        UZIP_CUDA_TRY(cudaFuncSetAttribute(mass_kernel<QT, FP8, DP, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem));
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    mass_kernel<QT, FP8, DP, TMA><<<p.grid, kMassThreads, C::kSmem, stream>>>(p, maps);
    UZIP_CUDA_TRY(cudaGetLastError());
    return UZIP_OK;
}

template <typename QT, bool FP8, int DP>
int launch_mass_as(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t stream) {
    using C = MassCfg<QT, FP8, DP>;
    const uint32_t chunks = (p.rows + C::kMaxN - 1) / C::kMaxN;
    p.mtiles = chunks;
    p.m = ((p.rows + chunks - 1) / chunks + 15) / 16 * 16;
    p.shift = 7;
    p.unit_cost = 5;
    static_assert(kMassTile == 1u << 7, "tile");
    p.grid = (uint32_t)sms;
    Maps maps{};
    if (maps_of(p, c, kMassTile, 2048, &maps)) return launch_mass_by<QT, FP8, DP, true>(p, maps, stream);
    return launch_mass_by<QT, FP8, DP, false>(p, maps, stream);
}

template <typename QT, bool FP8>
int launch_mass(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s) {
    if (p.cache.head_dim <= 64) return launch_mass_as<QT, FP8, 64>(p, c, sms, s);
    if (p.cache.head_dim <= 128) return launch_mass_as<QT, FP8, 128>(p, c, sms, s);
    return launch_mass_as<QT, FP8, 256>(p, c, sms, s);
}

}  // namespace uzkv
