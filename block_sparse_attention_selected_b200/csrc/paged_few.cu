// paged_few.cu -- paged attention for units of few query rows (single tokens, drafted
// tokens, one token's selected blocks): the transposed products.
//
// With a tile of 128 query rows per unit (paged_attn.cu) a single token's G rows lie in one
// warp's TMEM lanes: that warp alone works through 128 keys a row, and the tensor pipe
// multiplies rows that do not exist.  Here keys and value columns are the 128 rows of the
// products and the N = 16 query rows their columns:
//     S^T [128 keys x N] = K Q^T          O^T [D columns x N] += V^T P^T
// so a thread holds one key's scores of all N rows, the softmax of a tile is N values a
// thread on all four schedulers, and a product is N / 128 of the work.  P^T goes through
// shared memory (K-major, N rows of 128 keys).
//
// The reference m of a row (see paged_attn.cu) is common to the threads of a stream.  A tile
// in which no score passes m + kLazy needs no maximum at all: the warps only tell each other
// so.  Otherwise all rows' maxima are taken over the tile, and O^T and the sums rescaled.
//
// Units, pieces, scheduler and producer: paged_attn.cuh.  Two streams take the even and the
// odd key tiles; S^T, P^T and (over units) O^T are double-buffered, so that S^T of the next
// tiles and the epilogue of a unit run under the other products.
//
// What bounds it: memory, or what lies before it.  64 requests of one token (4 query heads per
// KV head, 512 to 32768 keys, 4.36 GB of K and V): 635 us, 6.9 TB/s.  One request of 8192 keys:
// 18 us, of which the data need 5; the rest is the scheduler's first piece and the
// first page lookup, each a chain of loads, and the merge.  Selected blocks of 64 requests: 62 us,
// 4.4 TB/s; a chunk of 512 tokens, 2.1 GB out of L2: 288 us, 7.5 TB/s, 26 bytes a cycle and SM
// over the whole call, near the 28 that the TMA unit takes in.  These two change by a few per cent
// with the size of the code (selected blocks of the chunk: 288 - 334 us with longer and longer
// wait loops), so what every wait carries is kept short.
// P^T is rounded to the type of V and l sums the unrounded weights, as in paged_attn.cu.
//
//   warps 0-7    softmax and epilogue: a warpgroup per stream, one thread per key of the tile
//                (per value column in the epilogue)
//   warp 8       TMA producer          warp 10  scheduler
//   warps 9, 11  MMA issuers, one per stream
#include <algorithm>

#include "paged_attn.cuh"

namespace nsa {
namespace {

constexpr int N = kFewRows;
constexpr int kFewThreads = 384;
constexpr int kFewSoftmax = 8;

template <int D>
struct alignas(1024) FewSmem {
    static constexpr int kHalves = D / 64;
    // 32 KB (D = 128) or 16 KB (D = 64) each; what fits next to Q and P^T
    static constexpr int kStages = D == 128 ? 6 : 12;
    static constexpr int kAhead = 2;          // S^T tiles of a stream ahead of its P V
    uint8_t q[2][kHalves][N * 128];           // [unit parity][64 columns][row]
    uint8_t pt[2][2][2][N * 128];             // [stream][buffer][64 keys][row]
    uint8_t kv[kStages][kHalves * kRegion];
    Piece ring[kRing];
    int list[kRing][kMaxTopk];
    float wmax[2][4][N];                      // [stream][warp][row] a tile's maxima
    float m[2][2][N];                         // [unit parity][stream][row]
    float l[2][2][4][N];                      // [unit parity][stream][warp][row]
    int flag[2][2][4];                        // [item parity][stream][warp] a maximum grew
    uint64_t ring_full[kRing], ring_empty[kRing];
    uint64_t q_full[2], q_empty[2];
    uint64_t kv_full[kStages], kv_empty[kStages];
    // [stream][buffer]: a stream may be two items, or two units, ahead of the one that waits
    uint64_t s_full[2][2], p_full[2][2], o_full[2][2], o_empty[2][2];
    uint64_t pv_done[2], meet[2];
    uint64_t xbar, drain;
    uint32_t tmem_base;
    int abort_flag, err;
    int loaded[3];                            // K tiles, V tiles and Qs that the producer asked for
};

// 8 and 16 fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld8_sync(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "{\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr) : "memory");
}

// Reduces v[0 .. 16) over the 32 lanes at 16 shuffles: at each of the first steps a lane keeps
// half of its values.  Lanes i and i + 16 end with the result of value i.
template <class Op>
__device__ __forceinline__ float transpose_reduce(float (&v)[N], int lane, Op op) {
#pragma unroll
    for (int n = N / 2; n >= 1; n >>= 1) {
        const bool up = lane & n;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, n));
        }
    }
    return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

template <int F16, int D, bool SEL>
__global__ void __launch_bounds__(kFewThreads, 1)
    k_paged_few(const Params P, const __grid_constant__ CUtensorMap qmap,
                const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using Smem = FewSmem<D>;
    constexpr int kHalves = Smem::kHalves, kStages = Smem::kStages;
    using Stages = Ring<2, kStages / 2, Smem::kAhead>;
    constexpr uint32_t kCols = 8 * N;             // TMEM: S^T [stream][buffer], O^T [stream][unit parity]
    extern __shared__ uint8_t smem_raw[];
    Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const PagedAttnArgs& p = P.a;
    // hardware warps 0-3 are 8-11 below: the issuers come first in the schedulers' order
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = (tid >> 5) < 4 ? kFewSoftmax + (tid >> 5) : (tid >> 5) - 4;
    const int cta = (int)blockIdx.x, grid = (int)gridDim.x;

    if (tid == 0) {
        S.abort_flag = 0;
        S.err = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.q_full[i], 1);
            mbar_init(&S.q_empty[i], 2);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&S.s_full[i][b], 1);
                mbar_init(&S.p_full[i][b], 4);
                mbar_init(&S.o_full[i][b], 1);
                mbar_init(&S.o_empty[i][b], kFewSoftmax);
            }
            mbar_init(&S.pv_done[i], 1);
            mbar_init(&S.meet[i], 4);
        }
        for (int i = 0; i < kStages; ++i) {
            // (a test: the first tile of K, place 0, waits for an arrival that never comes)
            mbar_init(&S.kv_full[i], i == 0 && cta == 0 && p.test_skip ? 2 : 1);
            mbar_init(&S.kv_empty[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&S.ring_full[i], 1);
            mbar_init(&S.ring_empty[i], 3 + kFewSoftmax);
        }
        mbar_init(&S.xbar, kFewSoftmax);
        mbar_init(&S.drain, 2);
        fence_barrier_init();
    }
    if (warp == 10 && lane == 0) {
        prefetch_tmap(&qmap);
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    release_dependents();
    depend();
    // (not before: a kernel that this one waits for may need the tensor memory)
    if (warp == 8) {
        __syncwarp();
        tmem_alloc(&S.tmem_base, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    const Waiter wait{&S.abort_flag, &S.err};

    if (warp == 8) {
        produce<SEL, 1, Stages>(S, P, wait, &qmap, &kmap, &vmap, lane);
    } else if (warp == 10) {
        schedule<SEL>(S, P, wait, P.tpt, cta, grid, lane);
    } else if (warp >= kFewSoftmax) {
        // ------------------------------------------------------------- MMA issuers
        const uint32_t elected = elect_one();
        constexpr uint32_t kIdescS = idesc_f16kind_f32(F16 != 0, 128, N, false, false);
        constexpr uint32_t kIdescO = idesc_f16kind_f32(F16 != 0, 128, N, true, false);
        using Kv = Tile<D>;
        constexpr uint32_t kTileU = kHalves * kRegion >> 4;
        constexpr uint32_t kStepU = 2 * Kv::kGroupU;     // 16 keys of V
        constexpr uint32_t kSmallU = (N * 128) >> 4;     // 64 columns of Q, 64 keys of P^T
        auto u = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
        const int st = (int)u(warp == 9 ? 0u : 1u);
        const uint32_t tS = u(tmem + st * 2u * N), tO = u(tmem + 4u * N + st * 2u * N);
        const uint32_t q_desc0 = u((uint32_t)smem_desc_sw128(smem_u32(S.q[0][0]), 16, 1024));
        const uint32_t k_desc0 = u((uint32_t)smem_desc_sw128(smem_u32(S.kv[0]), 16, 0));
        // V^T: 128 rows are two 64-column halves; with D = 64 the half is read twice and
        // lanes 64 - 127 of O^T repeat lanes 0 - 63
        const uint32_t v_desc0 = u((uint32_t)smem_desc_sw128(smem_u32(S.kv[0]), D == 128 ? 1024 : 0, 0));
        const uint32_t p_desc0 = u((uint32_t)smem_desc_sw128(smem_u32(S.pt[st][0][0]), 16, 1024));
        int at_s = -1, js = 0, js_end = 0, base_s = 0, count_s = 0, units_s = 0, items_s = 0;
        int at_o = -1, jo = 0, jo_end = 0, base_o = 0, count_o = 0, items_o = 0, sums = 0;
        bool first_o = true, ok = true, more_s = true, more_o = true;
        int lo_o = 0, hi_o = 0, tile0_o = 0;
        int qb = 0;
        auto first_tile = [&](int p0, int count) { return p0 + ((count & 1) ^ st); };
        // to the next S^T; everything it waits for (its buffer is free: P^T of the item two
        // before has been waited for).  more_s: there is one
        auto prepare_s = [&]() -> bool {
            while (more_s && js >= js_end) {
                if (!fetch_piece(S, wait, ++at_s)) return false;
                const Piece& k = S.ring[at_s % kRing];
                more_s = k.more != 0;
                const int p0 = k.p0, nt = k.p1 - p0;
                if (!more_s) break;
                qb = units_s & 1;
                ++units_s;
                js = first_tile(p0, count_s);
                js_end = p0 + nt;
                base_s = count_s - p0;
                count_s += nt;
                // (a unit without a tile for this stream is waited for as well, or this
                // issuer could be done with a later Q of the buffer before the other is with
                // this one)
                if (!wait(&S.q_full[qb], ((units_s - 1) >> 1) & 1)) return false;
                if (js >= js_end) mma_commit_e(&S.q_empty[qb], elected);
            }
            if (!more_s) return true;
            const auto to = Stages::k(base_s + js);
            return wait(&S.kv_full[to.stage], to.phase);
        };
        auto issue_s = [&]() {
            const int stg = Stages::k(base_s + js).stage, b = items_s & 1;
            const uint32_t a0 = u(k_desc0 + (uint32_t)stg * kTileU);
            const uint32_t b0 = u(q_desc0 + (uint32_t)qb * kHalves * kSmallU);
            const uint32_t d0 = u(tS + (uint32_t)b * N);
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
                mma_ss_hi(d0, a0 + (uint32_t)((x >> 2) * Kv::kHalfU + (x & 3) * 2), Kv::kDescHi,
                          b0 + (uint32_t)((x >> 2) * kSmallU + (x & 3) * 2), kSw128Sbo1024DescHi, kIdescS, x > 0 ? 1u : 0u,
                          elected);
            mma_commit_e(&S.s_full[st][b], elected);
            mma_commit_e(&S.kv_empty[stg], elected);
            ++items_s;
            js += 2;
            if (js >= js_end) mma_commit_e(&S.q_empty[qb], elected);
        };
        for (int i = 0; i < Smem::kAhead && ok; ++i) {
            ok = prepare_s();
            if (ok && more_s) issue_s();
        }
        while (ok) {
            while (more_o && jo >= jo_end) {
                if (at_o >= 0) release_piece(S, lane, at_o);
                if (!(ok = fetch_piece(S, wait, ++at_o))) break;
                const Piece& k = S.ring[at_o % kRing];
                more_o = k.more != 0;
                const int p0 = k.p0, nt = k.p1 - p0;
                if (!more_o) break;
                jo = first_tile(p0, count_o);
                jo_end = p0 + nt;
                base_o = count_o - p0;
                count_o += nt;
                lo_o = k.lo;
                hi_o = k.hi;
                tile0_o = k.tile0;
                first_o = true;
            }
            if (!ok || !more_o) break;
            const auto from = Stages::v(base_o + jo);
            const int stg = from.stage;
            if (!(ok = wait(&S.kv_full[stg], from.phase))) break;
            int l0, h0, l1, h1;               // the tile's visible columns
            if (SEL) {
                tile_cols<SEL>(P, S.ring[at_o % kRing], S.list[at_o % kRing], jo, l0, h0, l1, h1);
            } else {
                const int key0 = (tile0_o + jo) * kTileKeys;
                l0 = max(lo_o - key0, 0);
                h1 = min(hi_o - key0, 127);
                h0 = min(h1, 63);
                l1 = max(l0, 64);
            }
            const bool full = l0 == 0 && h0 == 63 && l1 == 64 && h1 == 127;
            if (!full) {   // clear the rows of the used 16-key steps that nobody may see
                uint8_t* v = S.kv[stg];
                auto clear = [&](int from, int to) { clear_rows<D>(v, from, to, lane); };
                if (l0 <= h0) { clear(l0 & ~15, l0); clear(h0 + 1, (h0 + 16) & ~15); }
                if (l1 <= h1) { clear(l1 & ~15, l1); clear(h1 + 1, (h1 + 16) & ~15); }
                fence_async_smem();
                __syncwarp();
            }
            // O^T's buffer: read out by the epilogue of the sum before the last
            if (first_o && sums > 1 && !(ok = wait(&S.o_empty[st][sums & 1], ((sums >> 1) - 1) & 1))) break;
            if (!(ok = prepare_s())) break;
            if (!(ok = wait(&S.p_full[st][items_o & 1], (items_o >> 1) & 1))) break;
            tc_fence_after();
            {
                const uint32_t a0 = u(v_desc0 + (uint32_t)stg * kTileU);
                const uint32_t b0 = u(p_desc0 + (uint32_t)(items_o & 1) * 2 * kSmallU);
                const uint32_t d0 = u(tO + (uint32_t)(sums & 1) * N);
                uint32_t acc = first_o ? 0u : 1u;
                if (full) {
#pragma unroll
                    for (int x = 0; x < kTileKeys / 16; ++x)
                        mma_ss_hi(d0, a0 + x * kStepU, Kv::kDescHi, b0 + (uint32_t)((x >> 2) * kSmallU + (x & 3) * 2),
                                  kSw128Sbo1024DescHi, kIdescO, x == 0 ? acc : 1u, elected);
                } else {
#pragma unroll 1
                    for (int x = 0; x < kTileKeys / 16; ++x) {
                        const bool use = x < 4 ? (l0 <= h0 && 16 * x + 15 >= l0 && 16 * x <= h0)
                                               : (l1 <= h1 && 16 * x + 15 >= l1 && 16 * x <= h1);
                        if (use) {
                            mma_ss_hi(d0, a0 + x * kStepU, Kv::kDescHi,
                                      b0 + (uint32_t)((x >> 2) * kSmallU + (x & 3) * 2), kSw128Sbo1024DescHi, kIdescO, acc,
                                      elected);
                            acc = 1u;
                        }
                    }
                }
            }
            first_o = false;
            mma_commit_e(&S.kv_empty[stg], elected);
            mma_commit_e(&S.pv_done[st], elected);
            jo += 2;
            ++items_o;
            if (jo >= jo_end) {
                mma_commit_e(&S.o_full[st][sums & 1], elected);
                ++sums;
            }
            if (more_s) issue_s();
        }
        mma_commit_e(&S.drain, elected);
        const long long start = clock64();
        while (!mbar_try_wait(&S.drain, 0) && clock64() - start < kWaitBudgetCycles) {}
    } else {
        // ------------------------------------------------------- softmax and epilogue
        const int st = warp >> 2, quad = warp & 3, key = quad * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + lane_off + (uint32_t)(st * 2 * N), tO = tmem + lane_off + 4u * N;
        const float c = p.scale_log2;
        // this key's place in P^T [64 keys][row]: row r adds (r >> 3) * 1024 + (r & 7) * 128
        // and the swizzle of its 16-byte chunk
        const uint32_t chunk = (uint32_t)((key & 63) >> 3);
        const uint32_t pt0 = smem_u32(S.pt[st][0][key >> 6]) + (uint32_t)(key & 7) * 2u;
        int items = 0, tiles = 0, units = 0, meets = 0;
        int o_next[2] = {0, 0};           // sums each stream has begun
        bool ok = true;
        auto meet = [&]() -> bool {           // the four warps of the stream
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.meet[st]);
            return wait(&S.meet[st], meets++ & 1);
        };
        // A finished unit's output.  It waits for the unit's last P V and for the other stream,
        // so it is left until the first tile of the next unit is on its way.
        struct Done { int at, par, n0, n1, c0, c1; };     // par: the unit's parity
        Done done{-1, 0, 0, 0, 0, 0};
        auto finish = [&]() -> bool {
            const Piece& k = S.ring[done.at % kRing];
            const int par = done.par, rows = k.ntok * p.G;
            bool fine = wait(&S.xbar, par);
            if (fine && done.n0 > 0) fine = wait(&S.o_full[0][done.c0 & 1], (done.c0 >> 1) & 1);
            if (fine && done.n1 > 0) fine = wait(&S.o_full[1][done.c1 & 1], (done.c1 >> 1) & 1);
            if (!fine) return false;
            tc_fence_after();
            // this thread: value column `key` of half of the rows (the other half: the other
            // warpgroup)
            const int slot = k.slot, tok0 = k.tok0, hq0 = k.g * p.G;
            const uint32_t o0 = tO + (uint32_t)((done.c0 & 1) * N), o1 = tO + (uint32_t)((2 + (done.c1 & 1)) * N);
            const int x = st * (N / 2);
            if (x < rows) {
                float a[8], b[8];
                tmem_ld8_sync(o0 + x, a);
                tmem_ld8_sync(o1 + x, b);
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const int r = x + y;
                    if (r >= rows) break;
                    const float m0 = S.m[par][0][r], m1 = S.m[par][1][r];
                    const float l0 = S.l[par][0][0][r] + S.l[par][0][1][r] + S.l[par][0][2][r] + S.l[par][0][3][r];
                    const float l1 = S.l[par][1][0][r] + S.l[par][1][1][r] + S.l[par][1][2][r] + S.l[par][1][3][r];
                    const float mm = fmaxf(m0, m1);
                    const float w0 = l0 != 0.f ? ex2_approx(m0 - mm) : 0.f;   // (a NaN sum stays one)
                    const float w1 = l1 != 0.f ? ex2_approx(m1 - mm) : 0.f;
                    const float ll = w0 * l0 + w1 * l1;
                    // a weight of 0 belongs to a sum that may never have been started
                    const float o = (w0 != 0.f ? w0 * a[y] : 0.f) + (w1 != 0.f ? w1 * b[y] : 0.f);
                    if (slot < 0) {
                        const int t = r / p.G, tok = tok0 + t, hq = hq0 + r - t * p.G;
                        const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : CUDART_NAN_F);
                        if (key < D) p.out[((size_t)tok * p.hq + hq) * D + key] = (uint16_t)pack2<F16>(o * inv, 0.f);
                        if (p.lse && key == 0)
                            p.lse[(size_t)hq * p.T + tok] =
                                ll == 0.f ? -CUDART_INF_F : (mm + log2f(ll)) * 0.69314718055994531f;
                    } else {
                        if (key < D) P.part_o[((size_t)slot * 128 + r) * D + key] = o;
                        if (key == 0) P.part_ml[(size_t)slot * 128 + r] = make_float2(mm, ll);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (done.n0 > 0) mbar_arrive(&S.o_empty[0][done.c0 & 1]);
                if (done.n1 > 0) mbar_arrive(&S.o_empty[1][done.c1 & 1]);
            }
            release_piece(S, lane, done.at);
            done.at = -1;
            return true;
        };
        for (int at = 0;; ++at) {
            if (!(ok = fetch_piece(S, wait, at))) break;
            const Piece& k = S.ring[at % kRing];
            if (!k.more) break;
            const int* list = S.list[at % kRing];
            const int rows = k.ntok * p.G, p0 = k.p0, p1 = k.p1, nt = p1 - p0;
            const int n0 = (nt + 1 - (tiles & 1)) >> 1, n1 = nt - n0;
            const int from = p0 + ((tiles & 1) ^ st);
            tiles += nt;
            float m[N], l[N];
#pragma unroll
            for (int r = 0; r < N; ++r) {
                m[r] = -CUDART_INF_F;
                l[r] = 0.f;
            }
            for (int j = from; j < p1; j += 2, ++items) {
                // rows [r0, r1) see this thread's key
                int r0 = 0, r1 = rows;
                if (SEL) {
                    int l0, h0, l1, h1;
                    tile_cols<SEL>(P, k, list, j, l0, h0, l1, h1);
                    if (key < 64 ? (key < l0 || key > h0) : (key < l1 || key > h1)) r1 = 0;
                } else {
                    // token t (position pos0 + t) sees key x iff pos0 + t - W < x <= pos0 + t
                    const int ahead = (k.tile0 + j) * kTileKeys + key - k.pos0;
                    r0 = ahead > 0 ? (ahead < k.ntok ? ahead * p.G : N) : 0;
                    if (p.swin > 0) {
                        const int t1 = ahead + p.swin;           // tokens below t1
                        r1 = t1 <= 0 ? 0 : (t1 < k.ntok ? t1 * p.G : rows);
                    }
                }
                if (!(ok = wait(&S.s_full[st][items & 1], (items >> 1) & 1))) break;
                tc_fence_after();
                float s[N];
                tmem_ld16_sync(tS + (uint32_t)((items & 1) * N), s);
                bool grow = false;
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    s[r] = r >= r0 && r < r1 ? s[r] * c : -CUDART_INF_F;
                    grow |= s[r] > m[r] + kLazy;
                }
                grow = __any_sync(0xffffffffu, grow);
                if (lane == 0) S.flag[items & 1][st][quad] = grow;
                if (!(ok = meet())) break;
                const int4 f = *reinterpret_cast<const int4*>(S.flag[items & 1][st]);
                if (f.x | f.y | f.z | f.w) {
                    // the tile's maximum of every row, over lanes and warps
                    float t[N];
#pragma unroll
                    for (int r = 0; r < N; ++r) t[r] = s[r];
                    const float top = transpose_reduce(t, lane, [](float a, float b) { return fmaxf(a, b); });
                    if (lane < N) S.wmax[st][quad][lane] = top;
                    if (!(ok = meet())) break;
                    // (O^T: the stream's last P V has to be complete)
                    if (j != from && !(ok = wait(&S.pv_done[st], (items - 1) & 1))) break;
                    tc_fence_after();
                    const uint32_t o0 = tO + (uint32_t)((st * 2 + (o_next[st] & 1)) * N);
                    float a[N], o[N];
#pragma unroll
                    for (int r = 0; r < N; ++r) {
                        const float mx = fmaxf(fmaxf(S.wmax[st][0][r], S.wmax[st][1][r]),
                                               fmaxf(S.wmax[st][2][r], S.wmax[st][3][r]));
                        const bool g = mx > m[r] + kLazy;
                        a[r] = g ? ex2_approx(m[r] - mx) : 1.f;     // m = -inf: 0
                        if (g) m[r] = mx;
                        l[r] *= a[r];
                    }
                    if (j != from) {
                        tmem_ld16_sync(o0, o);
#pragma unroll
                        for (int r = 0; r < N; ++r) o[r] *= a[r];
                        tmem_st16_sync(o0, o);
                    }
                }
                const uint32_t pt = pt0 + (uint32_t)(items & 1) * (2 * N * 128);
#pragma unroll
                for (int r = 0; r < N; r += 2) {
                    const float e0 = ex2_approx(s[r] - (m[r] == -CUDART_INF_F ? 0.f : m[r]));
                    const float e1 = ex2_approx(s[r + 1] - (m[r + 1] == -CUDART_INF_F ? 0.f : m[r + 1]));
                    l[r] += e0;
                    l[r + 1] += e1;
                    const uint32_t w = pack2<F16>(e0, e1);
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(
                                     pt + (r >> 3) * 1024u + (r & 7) * 128u + ((chunk ^ (r & 7)) << 4)),
                                 "h"((uint16_t)w) : "memory");
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(
                                     pt + ((r + 1) >> 3) * 1024u + ((r + 1) & 7) * 128u + ((chunk ^ ((r + 1) & 7)) << 4)),
                                 "h"((uint16_t)(w >> 16)) : "memory");
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.p_full[st][items & 1]);
                if (done.at >= 0 && !(ok = finish())) break;
            }
            if (!ok) break;
            if (done.at >= 0 && !(ok = finish())) break;     // (no tile of this unit for the stream)
            done = {at, units & 1, n0, n1, o_next[0], o_next[1]};
            // the rows' references and sums, for both streams' threads
            if (quad == 0 && lane == 0) {
#pragma unroll
                for (int r = 0; r < N; ++r) S.m[done.par][st][r] = m[r];
            }
            const float lsum = transpose_reduce(l, lane, [](float a, float b) { return a + b; });
            if (lane < N) S.l[done.par][st][quad][lane] = lsum;
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.xbar);
            o_next[0] += n0 > 0;
            o_next[1] += n1 > 0;
            ++units;
        }
        if (ok && done.at >= 0) finish();
    }

    // ---- teardown: every role has left its loop (all waits are bounded) and the issuers
    //      have drained their tensor-core work
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) {
        if (S.abort_flag) land_copies<1, Stages>(S, lane);
        tmem_dealloc(tmem, kCols);
    }
    if (tid == 0) finish_status(p.st, S.err, cta, grid);
}

template <int F16, int D, bool SEL>
cudaError_t launch(const Params& P, int grid, const CUtensorMap& qmap, const CUtensorMap& kmap,
                   const CUtensorMap& vmap, cudaStream_t stream) {
    const size_t smem = sizeof(FewSmem<D>) + 1024;
    cudaError_t e = cudaFuncSetAttribute(k_paged_few<F16, D, SEL>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_paged_few<F16, D, SEL>, grid, kFewThreads, smem, stream, P, qmap, kmap, vmap);
}

template <int F16, int D>
cudaError_t dispatch(const Params& P, int grid, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                     cudaStream_t stream) {
    return P.a.bidx ? launch<F16, D, true>(P, grid, q, k, v, stream)
                    : launch<F16, D, false>(P, grid, q, k, v, stream);
}

}  // namespace

cudaError_t launch_paged_few(const Params& P, int f16, int grid, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, cudaStream_t stream) {
    if (P.a.d == 64)
        return f16 ? dispatch<1, 64>(P, grid, q, k, v, stream) : dispatch<0, 64>(P, grid, q, k, v, stream);
    return f16 ? dispatch<1, 128>(P, grid, q, k, v, stream) : dispatch<0, 128>(P, grid, q, k, v, stream);
}

}  // namespace nsa
