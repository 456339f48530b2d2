// paged_attn.cu -- attention of new tokens over a paged K/V cache, over all of the
// visible keys or over the key blocks that each (token, KV head) selects.
//
// Mathematics: one pass over the visible keys of a tile of query rows, 128 keys at a
// time, S = Q K^T, P = 2^(c S - m), O += P V, with the running reference m of each row and
// the sum l of its weights (c = scale log2 e).  m follows the row's maximum lazily: O and
// l are rescaled only when the maximum has grown by more than 2^8 (kLazy), so that P stays
// below 2^8 and fp32 sums lose nothing.
//
// P is rounded to the 16-bit type of V for the second product, whose operands have one type: half
// a step (2^-9 in bf16) per weight, independent from key to key, which on rows of many like
// weights adds about as much as the rounding of the output does (relative error against 64 bits
// 2.3e-3, of the output's rounding alone 1.7e-3).  l sums the unrounded weights: it gives the lse
// too, which keeps 32 bits that way (error below 1e-7).  (The packed forward divides by the sum
// of the rounded weights and keeps a second sum for its lse: a row that one key dominates then
// has that key's V to one rounding, here to two.)
//
// (paged_attn.cuh: units, their division among the CTAs, the scheduler and the producer.)
// Two streams of (S, P, O) alternate on the tensor pipe, so that one stream's softmax runs
// under the other's products:
//   NQ = 2  two tiles of 128 query rows over the same key tiles (long chunks);
//   NQ = 1  one tile of query rows, even and odd key tiles, joined when the unit ends
//           (single tokens and short chunks: K and V are read once from memory, which
//           bounds them).
//
//   warps 0-7    softmax and epilogue: a warpgroup per stream, one thread per query row
//   warp 8       TMA producer: Q tiles, K and V tiles page by page through the block table
//   warps 9, 11  MMA issuers, one per stream
//   warp 10      scheduler: walks the CTA's pieces of work ahead of the others and hands
//                them over through a ring in shared memory
//
// What bounds it.  A chunk of 2048 tokens behind 30720 cached ones (32 query over 8 KV heads,
// d = 128) takes 917 us, 1.16 PFLOP/s, 70 % of the measured burst rate of a library product of
// bf16 matrices, in runs too short for the power limit; a call among others takes 1072 - 1092 us,
// 0.98 PFLOP/s, 71 % of that product's sustained rate (the clock falls).  Per pair of key tiles (four products of 512 tensor
// cycles) a stream's chain is about 1900 cycles of softmax (S from TMEM 310, maximum 350,
// exponentials 1200 of which the special-function unit needs 1024) and 1000 - 1700 of its two
// products.  Measured and not taken: four softmax warpgroups with two threads a row (1016 us:
// the two meet once a tile, and TMEM loads queue); every 8th, 4th or 2nd pair of exponentials
// by polynomial (972 - 1285 us); S in halves of 64 keys (fewer cycles, but Q is read twice a
// tile and the clock falls: 1010 us); weights formed before the maximum is known (1040 us);
// one issuer warp for both streams (957 us); the special warps last in the block (1170 us).
// 16 requests of 3 - 9 tokens on pages of 16: 55 us, 4.1 TB/s; long caches 5.8 TB/s (pages of 64:
// 6.6), bound by the issue of TMA boxes, one a page.
// Registers: 4 bytes a thread are spilled; 20, read back at 92 places, in the instances for
// selected blocks of more than 16 query heads per KV head.
#include <algorithm>
#include <type_traits>

#include "paged_attn.cuh"

namespace nsa {
namespace {

constexpr int kPaThreads = 384;
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kPaThreads * 168, "registers of the launch");
template <int D>
struct alignas(1024) PaSmem {
    static constexpr int kHalves = D / 64;
    static constexpr int kStages = D == 128 ? 4 : 8;
    uint8_t q[2][kHalves][kRegion];           // NQ = 2: the unit's two tiles; NQ = 1: two units
    uint8_t kv[kStages][kHalves * kRegion];   // K and V tiles in the order the issuer uses them
    float2 xch[2][2][128];                    // NQ = 1: [unit parity][stream][row] (m, l)
    Piece ring[kRing];                        // the scheduler's pieces, in order
    int list[kRing][kMaxTopk];                // selected blocks: the valid ones of each
    uint64_t ring_full[kRing], ring_empty[kRing];
    uint64_t q_full[2], q_empty[2];
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_empty[2];
    uint64_t xbar, drain;
    uint32_t tmem_base;
    int abort_flag, err;
    int loaded[3];                            // K tiles, V tiles and Qs that the producer asked for
};

template <int N>
__device__ __forceinline__ void set_regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int F16, int D, int NQ, bool SEL>
__global__ void __launch_bounds__(kPaThreads, 1)
    k_paged_attn(const Params P, const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using Smem = PaSmem<D>;
    constexpr int kHalves = Smem::kHalves, kStages = Smem::kStages;
    using Stages = Ring<3 - NQ, kStages / (3 - NQ), 1>;
    extern __shared__ uint8_t smem_raw[];
    Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const PagedAttnArgs& p = P.a;
    // roles: hardware warps 0-3 are 8-11 below, so that the issuer is not the last its
    // scheduler picks
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = (tid >> 5) < 4 ? kSoftmaxWarps + (tid >> 5) : (tid >> 5) - 4;
    const int cta = (int)blockIdx.x, grid = (int)gridDim.x;

    if (tid == 0) {
        S.abort_flag = 0;
        S.err = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.q_full[i], 1);
            mbar_init(&S.q_empty[i], 2);
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.p_half[i], 4);
            mbar_init(&S.p_full[i], 4);
            mbar_init(&S.o_full[i], 1);
            mbar_init(&S.o_empty[i], NQ == 2 ? 4 : 8);
        }
        for (int i = 0; i < kStages; ++i) {
            // (a test: the first tile of K, place 0, waits for an arrival that never comes)
            mbar_init(&S.kv_full[i], i == 0 && cta == 0 && p.test_skip ? 2 : 1);
            mbar_init(&S.kv_empty[i], NQ);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&S.ring_full[i], 1);
            mbar_init(&S.ring_empty[i], 3 + kSoftmaxWarps);   // producer, issuers, softmax
        }
        mbar_init(&S.xbar, kSoftmaxWarps);
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
        tmem_alloc(&S.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    const Waiter wait{&S.abort_flag, &S.err};
    auto fetch = [&](int i) -> bool { return fetch_piece(S, wait, i); };
    auto release = [&](int i) { release_piece(S, lane, i); };

    // setmaxnreg at the head of each role: the compiler gives the code behind it that many
    if (warp >= kSoftmaxWarps) {
        set_regs_dec<kOtherRegs>();
        if (warp == 8) {
            produce<SEL, NQ, Stages>(S, P, wait, &qmap, &kmap, &vmap, lane);
        } else if (warp != 10) {
            // ------------------------------------------------------------- MMA issuers
            // Warp 9 issues for stream 0, warp 11 for stream 1.  A stream's next S follows its
            // P V on the in-order tensor pipe, which is what lets P share the columns of S.  The
            // 16 MMAs of an item (a key tile of a stream) are 1024 cycles of tensor work; next to
            // the busy softmax warps the code around them takes about as long, hence a warp per
            // stream, everything but P waited for first, addresses that every lane holds through
            // u() (the compiler then keeps them and all offsets in uniform registers), and a
            // piece's fields read once.
            const uint32_t elected = elect_one();
            constexpr uint32_t kIdescS = idesc_f16kind_f32(F16 != 0, 128, kTileKeys, false, false);
            constexpr uint32_t kIdescO = idesc_f16kind_f32(F16 != 0, 128, D, false, true);
            using Kv = Tile<D>;
            constexpr uint32_t kHalfU = kRegion >> 4, kTileU = kHalves * kHalfU;
            constexpr uint32_t kStepU = 2 * Kv::kGroupU;     // 16 keys of V
            constexpr int step = NQ == 2 ? 1 : 2;
            auto u = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
            const int st = (int)u(warp == 9 ? 0u : 1u);
            const uint32_t tS = u(tmem + st * 128u), tO = u(tmem + 256u + st * 128u);
            const uint32_t q_desc0 = u((uint32_t)smem_desc_sw128(smem_u32(S.q[0][0]), 16, 1024));
            const uint32_t k_desc0 = u((uint32_t)smem_desc_sw128(smem_u32(S.kv[0]), 16, 0));
            const uint32_t v_desc0 = u((uint32_t)smem_desc_sw128(smem_u32(S.kv[0]), 1024, 0));
            uint64_t *const s_full = &S.s_full[st], *const p_half = &S.p_half[st], *const p_full = &S.p_full[st];
            uint64_t *const o_full = &S.o_full[st],
                     *const o_empty = &S.o_empty[st];
            // two cursors over the pieces: the next S and the next P V; tile numbers over all
            // pieces give the stages
            int at_s = -1, js = 0, js_end = 0, base_s = 0, units_s = 0;
            int at_o = -1, jo = 0, jo_end = 0, base_o = 0;
            int count_s = 0, count_o = 0;     // key tiles of the pieces so far, both streams
            bool rows_s = true, rows_o = true;   // the unit has rows in this stream's tile
            int qb = 0;
            bool first_o = true;
            int lo_o = 0, hi_o = 0, tile0_o = 0;
            int sums = 0, items = 0;          // sums completed, P V items
            bool ok = true, more_s = true, more_o = true;
            auto first_tile = [&](int p0, int count) { return NQ == 2 ? p0 : p0 + ((count & 1) ^ st); };
            // to the next S; everything it waits for.  more_s: there is one
            auto prepare_s = [&]() -> bool {
                while (more_s && js >= js_end) {
                    if (!fetch(++at_s)) return false;
                    const Piece& k = S.ring[at_s % kRing];
                    more_s = k.more != 0;
                    const int p0 = k.p0, nt = k.p1 - p0;
                    if (!more_s) break;
                    qb = NQ == 2 ? 0 : units_s & 1;
                    ++units_s;
                    js = first_tile(p0, count_s);
                    js_end = p0 + nt;
                    base_s = count_s - p0;
                    count_s += nt;
                    rows_s = NQ == 1 || st == 0 || k.ntok > P.tpt;
                    // (a unit without a tile for this stream is waited for as well, or this
                    // issuer could be done with a later Q of the buffer before the other is with
                    // this one)
                    const int use = NQ == 2 ? units_s - 1 : (units_s - 1) >> 1;
                    if (!wait(&S.q_full[qb], use & 1)) return false;
                    if (js >= js_end) mma_commit_e(&S.q_empty[qb], elected);
                }
                if (!more_s) return true;
                const auto to = Stages::k(base_s + js);
                return wait(&S.kv_full[to.stage], to.phase);
            };
            auto issue_s = [&]() {
                const int stg = Stages::k(base_s + js).stage;
                const uint32_t a0 = u(q_desc0 + (uint32_t)(NQ == 2 ? st : qb) * kTileU);
                const uint32_t b0 = u(k_desc0 + (uint32_t)stg * kTileU);
                if (rows_s) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        mma_ss_hi(tS, a0 + (uint32_t)((x >> 2) * kHalfU + (x & 3) * 2), kSw128Sbo1024DescHi,
                                  b0 + (uint32_t)((x >> 2) * Kv::kHalfU + (x & 3) * 2), Kv::kDescHi, kIdescS,
                                  x > 0 ? 1u : 0u, elected);
                    }
                }
                mma_commit_e(s_full, elected);
                mma_commit_e(&S.kv_empty[stg], elected);
                js += step;
                if (js >= js_end) mma_commit_e(&S.q_empty[qb], elected);
            };
            ok = prepare_s();
            if (ok && more_s) issue_s();
            while (ok) {
                while (more_o && jo >= jo_end) {
                    if (at_o >= 0) release(at_o);
                    if (!(ok = fetch(++at_o))) break;
                    const Piece& k = S.ring[at_o % kRing];
                    more_o = k.more != 0;
                    const int p0 = k.p0, nt = k.p1 - p0;
                    if (!more_o) break;
                    jo = first_tile(p0, count_o);
                    jo_end = p0 + nt;
                    base_o = count_o - p0;
                    count_o += nt;
                    rows_o = NQ == 1 || st == 0 || k.ntok > P.tpt;
                    lo_o = k.lo;
                    hi_o = k.hi;
                    tile0_o = k.tile0;
                    first_o = true;
                }
                if (!ok || !more_o) break;
                const auto from = Stages::v(base_o + jo);
                const int stg = from.stage;
                if (!(ok = wait(&S.kv_full[stg], from.phase))) break;
                // the tile's visible columns; all of them but at a piece's ends
                int l0, h0, l1, h1;
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
                if (!full) {
                    // clear the rows of the used 16-key steps that nobody may see (NQ = 2: both
                    // issuers do, each before its own products)
                    uint8_t* v = S.kv[stg];
                    auto clear = [&](int from, int to) { clear_rows<D>(v, from, to, lane); };
                    if (l0 <= h0) { clear(l0 & ~15, l0); clear(h0 + 1, (h0 + 16) & ~15); }
                    if (l1 <= h1) { clear(l1 & ~15, l1); clear(h1 + 1, (h1 + 16) & ~15); }
                    fence_async_smem();
                    __syncwarp();
                }
                if (first_o && sums > 0 && !(ok = wait(o_empty, (sums - 1) & 1))) break;
                if (!(ok = prepare_s())) break;
                const uint32_t b0 = u(v_desc0 + (uint32_t)stg * kTileU);
                uint32_t acc = first_o ? 0u : 1u;
                if (!(ok = wait(p_half, items & 1))) break;
                tc_fence_after();
                if (rows_o && full) {         // the first 64 keys while the rows work on the others
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        mma_ts_hi(tO, tS + x * 8u, b0 + x * kStepU, Kv::kDescHi, kIdescO, x == 0 ? acc : 1u, elected);
                }
                if (!(ok = wait(p_full, items & 1))) break;
                tc_fence_after();
                if (rows_o && full) {
#pragma unroll
                    for (int x = 4; x < 8; ++x)
                        mma_ts_hi(tO, tS + x * 8u, b0 + x * kStepU, Kv::kDescHi, kIdescO, 1u, elected);
                } else if (rows_o) {
#pragma unroll 1
                    for (int x = 0; x < kTileKeys / 16; ++x) {
                        const bool use = x < 4 ? (l0 <= h0 && 16 * x + 15 >= l0 && 16 * x <= h0)
                                               : (l1 <= h1 && 16 * x + 15 >= l1 && 16 * x <= h1);
                        if (use) {
                            mma_ts_hi(tO, tS + x * 8u, b0 + x * kStepU, Kv::kDescHi, kIdescO, acc, elected);
                            acc = 1u;
                        }
                    }
                }
                first_o = false;
                mma_commit_e(&S.kv_empty[stg], elected);
                jo += step;
                ++items;
                if (jo >= jo_end) {               // the stream's last item of the unit: O is complete
                    mma_commit_e(o_full, elected);
                    ++sums;
                }
                if (more_s) issue_s();
            }
            mma_commit_e(&S.drain, elected);
            {
                const long long start = clock64();
                while (!mbar_try_wait(&S.drain, 0) && clock64() - start < kWaitBudgetCycles) {}
            }
        } else {
            schedule<SEL>(S, P, wait, P.tpu, cta, grid, lane);
        }
    } else {
        set_regs_inc<kSoftmaxRegs>();
        // ------------------------------------------------------- softmax and epilogue
        const int st = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + lane_off + (uint32_t)st * 128u, tO = tmem + lane_off + 256u;
        const int rt = row / p.G, head = row - rt * p.G;
        const float c = p.scale_log2;
        int items = 0;                    // this stream's items so far
        int tiles = 0;                    // NQ = 1: key tiles so far, both streams
        int units = 0;
        int o_cnt[2] = {0, 0};            // sums each stream has completed
        bool ok = true;
        for (int at = 0;; ++at) {
            if (!(ok = fetch(at))) break;
            const Piece& k = S.ring[at % kRing];
            if (!k.more) break;
            const int* list = S.list[at % kRing];
            const int ti = NQ == 2 ? st * P.tpt + rt : rt;         // token within the unit
            const bool valid = rt < P.tpt && ti < k.ntok;
            const int pos = k.pos0 + ti;
            const int row_lo = !SEL && p.swin > 0 ? max(0, pos - p.swin + 1) : 0;
            const bool active = __any_sync(0xffffffffu, valid);
            const int p0 = k.p0, p1 = k.p1, nt = p1 - p0;
            float m = -CUDART_INF_F, l = 0.f;
            // NQ = 1: key tiles of the piece alternate between the streams, from where the
            // last unit left off
            const int step = NQ == 2 ? 1 : 2;
            const int from = NQ == 2 ? p0 : p0 + ((tiles & 1) ^ st);
            for (int j = from; j < p1; j += step, ++items) {
                if (!(ok = wait(&S.s_full[st], items & 1))) break;
                if (active) {
                    tc_fence_after();
                    float s[128];
                    tmem_ld64_sync(tS, s);
                    tmem_ld64_sync(tS + 64, s + 64);
                    int l0, h0, l1, h1;   // this row's visible columns
                    if (SEL) {
                        tile_cols<SEL>(P, k, list, j, l0, h0, l1, h1);
                    } else {
                        const int key0 = (k.tile0 + j) * kTileKeys;
                        l0 = l1 = valid ? row_lo - key0 : 0;
                        h0 = h1 = valid ? pos - key0 : 127;
                    }
                    if (__any_sync(0xffffffffu, l0 > 0 || h0 < 63 || l1 > 64 || h1 < 127)) {
#pragma unroll
                        for (int x = 0; x < 64; ++x) {
                            if (x < l0 || x > h0) s[x] = -CUDART_INF_F;
                            if (x + 64 < l1 || x + 64 > h1) s[x + 64] = -CUDART_INF_F;
                        }
                    }
                    float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int x = 0; x < 128; x += 8)
#pragma unroll
                        for (int y = 0; y < 4; ++y) mx[y] = fmax3(mx[y], s[x + 2 * y], s[x + 2 * y + 1]);
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                    const bool grow = valid && top > m + kLazy;
                    if (__any_sync(0xffffffffu, grow)) {
                        const float a = grow ? ex2_approx(m - top) : 1.f;   // m = -inf: 0
                        if (grow) m = top;
                        l *= a;
                        if (j != from) {
                            // (the products before this S, P V of the last tile among them,
                            // are complete)
#pragma unroll 1
                            for (int x = 0; x < D; x += 16) {
                                float o[16];
                                tmem_ld16_sync(tO + (uint32_t)(st * 128 + x), o);
#pragma unroll
                                for (int y = 0; y < 16; ++y) o[y] *= a;
                                tmem_st16_sync(tO + (uint32_t)(st * 128 + x), o);
                            }
                        }
                    }
                    const float mm = m == -CUDART_INF_F ? 0.f : m;
                    const float2 c2 = make_float2(c, c), m2 = make_float2(-mm, -mm);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[32];
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            float2 e = fma2(make_float2(s[64 * h + 2 * x], s[64 * h + 2 * x + 1]), c2, m2);
                            e.x = ex2_approx(e.x);
                            e.y = ex2_approx(e.y);
                            sum[x & 1] = add2(sum[x & 1], e);
                            pk[x] = pack2<F16>(e.x, e.y);
                        }
                        tmem_st32_sync(tS + 32 * h, pk);
                        tc_fence_before();
                        if (h == 0) {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&S.p_half[st]);
                        }
                    }
                    const float2 t2 = add2(sum[0], sum[1]);
                    l += t2.x + t2.y;
                }
                __syncwarp();
                if (lane == 0) {
                    if (!active) mbar_arrive(&S.p_half[st]);
                    mbar_arrive(&S.p_full[st]);
                }
            }
            if (!ok) break;
            const int n0 = NQ == 2 ? nt : (nt + 1 - (tiles & 1)) >> 1, n1 = NQ == 2 ? nt : nt - n0;
            tiles += nt;
            float w0 = 0.f, w1 = 0.f;         // weights of the streams' sums
            if (NQ == 2) {
                if (!(ok = wait(&S.o_full[st], o_cnt[st]++ & 1))) break;
            } else {
                S.xch[units & 1][st][row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.xbar);
                ok = wait(&S.xbar, units & 1);
                if (ok && n0 > 0) ok = wait(&S.o_full[0], o_cnt[0]++ & 1);
                if (ok && n1 > 0) ok = wait(&S.o_full[1], o_cnt[1]++ & 1);
                if (!ok) break;
                const float2 a = S.xch[units & 1][0][row], b = S.xch[units & 1][1][row];
                m = fmaxf(a.x, b.x);
                w0 = a.y != 0.f ? ex2_approx(a.x - m) : 0.f;   // (a NaN sum stays one)
                w1 = b.y != 0.f ? ex2_approx(b.x - m) : 0.f;
                l = w0 * a.y + w1 * b.y;
            }
            tc_fence_after();
            const int tok = k.tok0 + ti, hq = k.g * p.G + head;
            const int slot = k.slot;
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : CUDART_NAN_F);
            // NQ = 1: each warpgroup takes half of the columns of every row
            constexpr int kCols = NQ == 2 ? D : D / 2;
            const int col0 = NQ == 2 ? 0 : st * kCols;
            const size_t part = (size_t)slot * (NQ * 128) + (NQ == 2 ? st * 128 : 0) + row;
            if (active) {
#pragma unroll 1
                for (int x = col0; x < col0 + kCols; x += 16) {
                    float o[16];
                    if (NQ == 2) {
                        tmem_ld16_sync(tO + (uint32_t)(st * 128 + x), o);
                    } else {
                        // a weight of 0 belongs to a sum that may never have been started
                        float o1[16];
                        tmem_ld16_sync(tO + (uint32_t)x, o);
                        tmem_ld16_sync(tO + (uint32_t)(128 + x), o1);
#pragma unroll
                        for (int y = 0; y < 16; ++y)
                            o[y] = (w0 != 0.f ? w0 * o[y] : 0.f) + (w1 != 0.f ? w1 * o1[y] : 0.f);
                    }
                    if (l == 0.f) {
#pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] = 0.f;
                    }
                    if (!valid) continue;
                    if (slot < 0) {
                        uint4* dst = reinterpret_cast<uint4*>(p.out + ((size_t)tok * p.hq + hq) * D + x);
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            dst[y] = make_uint4(pack2<F16>(o[8 * y] * inv, o[8 * y + 1] * inv),
                                                pack2<F16>(o[8 * y + 2] * inv, o[8 * y + 3] * inv),
                                                pack2<F16>(o[8 * y + 4] * inv, o[8 * y + 5] * inv),
                                                pack2<F16>(o[8 * y + 6] * inv, o[8 * y + 7] * inv));
                    } else {
                        float4* dst = reinterpret_cast<float4*>(P.part_o + part * D + x);
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            dst[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                    }
                }
                if (valid && col0 == 0) {
                    if (slot >= 0)
                        P.part_ml[part] = make_float2(m, l);
                    else if (p.lse)
                        p.lse[(size_t)hq * p.T + tok] =
                            l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (NQ == 2) {
                    mbar_arrive(&S.o_empty[st]);
                } else {
                    if (n0 > 0) mbar_arrive(&S.o_empty[0]);
                    if (n1 > 0) mbar_arrive(&S.o_empty[1]);
                }
            }
            ++units;
            release(at);
        }
    }

    // ---- teardown: every role has left its loop (all waits are bounded) and the issuer
    //      has drained its tensor-core work
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) {
        if (S.abort_flag) land_copies<NQ, Stages>(S, lane);
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0) finish_status(p.st, S.err, cta, grid);
}

// Joins the partial results of the unit that CTA blockIdx.x left open, in the order of the
// pieces.  One warp per row: lane i weighs piece i of each batch of 32, then all lanes add
// the pieces' columns, kBatch pieces' loads in flight: eight for units of one tile of rows,
// which many CTAs share (one token, 8192 keys: 18.4 us; four: 19.4), four for two tiles of rows,
// mostly cut once (a chunk of 512 behind 3584: 64 us a call; two: 65, eight: 71).
template <int F16, int D, int kBatch>
__global__ void __launch_bounds__(256) k_paged_merge(const Params P, int rows_per_piece) {
    release_dependents();
    depend();
    const PagedAttnArgs& p = P.a;
    const int4 d = P.desc[blockIdx.x];
    if (d.w < 0) return;
    const int lane = threadIdx.x & 31, first = blockIdx.x, np = d.w - first + 1;
    // piece 0 lies in slot 1 of CTA first, piece i in slot 0 of CTA first + i
    auto at = [&](int i, int row) -> size_t {
        return (size_t)(2 * (first + i) + (i == 0 ? 1 : 0)) * rows_per_piece + row;
    };
    constexpr int kV = D / 32;
    using Vec = typename std::conditional<kV == 4, float4, float2>::type;
    for (int y = blockIdx.y * 8 + (threadIdx.x >> 5); y < d.y * p.G; y += gridDim.y * 8) {
        const int ti = y / p.G, h = y - ti * p.G;
        const int row = (ti / P.tpt) * 128 + (ti % P.tpt) * p.G + h;
        float m = -CUDART_INF_F;
        for (int i = lane; i < np; i += 32) {
            const float2 ml = P.part_ml[at(i, row)];
            if (ml.y != 0.f) m = fmaxf(m, ml.x);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float acc[kV] = {}, l = 0.f;
        for (int b = 0; b < np; b += 32) {
            float w = 0.f;
            if (b + lane < np) {
                const float2 ml = P.part_ml[at(b + lane, row)];
                if (ml.y != 0.f) {
                    w = ex2_approx(ml.x - m);
                    l += w * ml.y;
                }
            }
            const int n = min(32, np - b);
            for (int c = 0; c < n; c += kBatch) {
                Vec o[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    o[i] = *reinterpret_cast<const Vec*>(P.part_o + at(b + min(c + i, n - 1), row) * D + lane * kV);
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const float wi = __shfl_sync(0xffffffffu, w, (c + i) & 31);
                    if (c + i < n) {
                        const float* e = reinterpret_cast<const float*>(&o[i]);
#pragma unroll
                        for (int x = 0; x < kV; ++x) acc[x] += wi * e[x];
                    }
                }
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : CUDART_NAN_F);
        const int tok = d.x + ti, hq = d.z * p.G + h;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + ((size_t)tok * p.hq + hq) * D + lane * kV);
#pragma unroll
        for (int x = 0; x < kV / 2; ++x) dst[x] = pack2<F16>(acc[2 * x] * inv, acc[2 * x + 1] * inv);
        if (p.lse && lane == 0)
            p.lse[(size_t)hq * p.T + tok] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
    }
}

bool encode(CUtensorMap* map, bool f16, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
    auto enc = get_encode_fn();
    if (!enc) return false;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
               const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int F16, int D, int NQ, bool SEL>
cudaError_t launch(const Params& P, int grid, const CUtensorMap& qmap, const CUtensorMap& kmap,
                   const CUtensorMap& vmap, cudaStream_t stream) {
    const size_t smem = sizeof(PaSmem<D>) + 1024;
    cudaError_t e = cudaFuncSetAttribute(k_paged_attn<F16, D, NQ, SEL>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_paged_attn<F16, D, NQ, SEL>, grid, kPaThreads, smem, stream, P, qmap, kmap, vmap);
}

template <int kBatch>
cudaError_t merge(const Params& P, int f16, int grid, int rows_per_piece, cudaStream_t stream) {
    auto* kernel = P.a.d == 64 ? (f16 ? k_paged_merge<1, 64, kBatch> : k_paged_merge<0, 64, kBatch>)
                               : (f16 ? k_paged_merge<1, 128, kBatch> : k_paged_merge<0, 128, kBatch>);
    const dim3 blocks((unsigned)grid, (unsigned)std::min(rows_per_piece / 32, (P.a.G * P.tpu + 7) / 8));
    return launch_dependent(kernel, blocks, 256, 0, stream, P, rows_per_piece);
}

template <int F16, int D>
cudaError_t dispatch(const Params& P, bool two, int grid, const CUtensorMap& q, const CUtensorMap& k,
                     const CUtensorMap& v, cudaStream_t stream) {
    if (P.a.bidx) return launch<F16, D, 1, true>(P, grid, q, k, v, stream);
    return two ? launch<F16, D, 2, false>(P, grid, q, k, v, stream)
               : launch<F16, D, 1, false>(P, grid, q, k, v, stream);
}

// Two tiles of query rows per unit where the batch has more than one tile of rows per
// request and KV head on average.
bool two_tiles(const PagedAttnArgs& p) { return (long long)p.T * p.G > 128ll * p.R; }

// The transposed products for units of few query rows: up to kFewRows rows of a token's query
// heads (selected blocks), or of a request's new tokens on average.  Measured against tiles of
// 128 rows: 64 requests of one token, 4 rows a unit, 634 against 662 us; 8 rows, 16 selected
// blocks, 67 against 67 us, a chunk of 512 such tokens 305 against 349 us.  The same kernel
// with 32 rows lost (16 requests of 3 - 9 tokens, 24 rows on average: 92 against 66 us): its
// Q and P^T leave room for two thirds of the K / V stages only.
// Both rules go by the batch's average, padding rows included, since the lengths are on the
// device: a batch of single tokens and one chunk has one kernel for both, at a price.  32 query
// over 8 KV heads, contexts to 16384, the chunk's 32768: 63 tokens and a chunk of 128 773 us
// (apart 363 + 94), 255 and 512 2959 us (1286 + 258), 63 and 2048 1549 us (341 + 1043).  A server
// that has the lengths on the host makes two calls.
bool few_rows(const PagedAttnArgs& p) {
    return (p.bidx ? p.G : std::max<long long>(p.G, (long long)p.T * p.G / p.R)) <= kFewRows;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t paged_attn_workspace(int d) {
    // status, descriptors, and two open units of 256 rows per CTA
    const size_t pieces = 2 * (size_t)kMaxStatusCtas;
    return align256(sizeof(DevStatus)) + align256(kMaxStatusCtas * sizeof(int4)) +
           align256(pieces * 256 * sizeof(float2)) + pieces * 256 * d * sizeof(float);
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int f16, int num_sms, cudaStream_t stream) {
    Params P{};
    P.a = a;
    uint8_t* ws = reinterpret_cast<uint8_t*>(a.st) + align256(sizeof(DevStatus));
    const size_t pieces = 2 * (size_t)kMaxStatusCtas;
    P.desc = reinterpret_cast<int4*>(ws);
    ws += align256(kMaxStatusCtas * sizeof(int4));
    P.part_ml = reinterpret_cast<float2*>(ws);
    P.part_o = reinterpret_cast<float*>(ws + align256(pieces * 256 * sizeof(float2)));
    const bool sel = a.bidx != nullptr;
    const bool few = few_rows(a);
    const bool two = !few && !sel && two_tiles(a);
    P.tpt = sel ? 1 : (few ? kFewRows : kTileRows) / a.G;
    P.tpu = two ? 2 * P.tpt : P.tpt;
    // A box is the keys of a page that a tile or block holds, in one dimension of 8-key groups
    // over all pages.  Pages that are no multiple of 8 keys apart go by boxes of 8 keys.
    const long long group = 8 * a.token_stride;
    const bool whole = group > 0 && (a.num_pages == 1 || (a.page_stride % group == 0 && a.page_stride / group >= a.ps / 8));
    const long long per_page = !whole ? 0 : a.num_pages == 1 ? a.ps / 8 : a.page_stride / group;
    P.page_groups = (per_page + 1) * (a.num_pages + 1ll) < (1ll << 31) ? (int)per_page : 0;
    P.box_rows = P.page_groups ? std::min(a.ps, sel ? std::min(a.bs, kTileKeys) : kTileKeys) : 8;
    int grid = std::min(num_sms, kMaxStatusCtas);
    if (sel) {
        P.cost_sel = (a.topk * a.bs + kTileKeys - 1) / kTileKeys + kUnitCost;
        const long long units = (long long)a.T * a.hkv, line = units * P.cost_sel;
        grid = (int)std::min<long long>(grid, line);
        // (512 units of 8 tiles on 148 SMs: 63 us whole, 67 us cut; 8 such units: cut)
        P.whole_sel = (units + grid - 1) / grid * P.cost_sel <= (line + grid - 1) / grid + kMergeCost;
    }
    CUtensorMap qmap, kmap, vmap;
    const cuuint64_t qdims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.hq, (cuuint64_t)a.T};
    // (a dimension of one element may have any stride; the map wants multiples of 16 bytes)
    auto stride = [&](long long elems, long long size) {
        return (cuuint64_t)(size > 1 ? elems : a.d) * 2;
    };
    const cuuint64_t qstr[2] = {stride(a.q_head_stride, a.hq), stride(a.q_token_stride, a.T)};
    const cuuint32_t qbox[3] = {64, (cuuint32_t)a.G, (cuuint32_t)P.tpt};
    // (64 columns, keys, halves, 8-key groups, heads) or (64 columns, keys, halves, heads, pages)
    const bool by_group = P.page_groups > 0;
    const cuuint64_t halves = a.d / 64, heads = a.hkv, pages = a.num_pages;
    const cuuint64_t groups = (pages - 1) * P.page_groups + a.ps / 8;
    const cuuint64_t kdims[5] = {64, (cuuint64_t)(by_group ? 8 : a.ps), halves, by_group ? groups : heads,
                                 by_group ? heads : pages};
    const cuuint64_t head_bytes = stride(a.head_stride, a.hkv);
    const cuuint64_t kstr[4] = {stride(a.token_stride, a.ps), 128, by_group ? (cuuint64_t)group * 2 : head_bytes,
                                by_group ? head_bytes : stride(a.page_stride, a.num_pages)};
    const cuuint32_t kbox[5] = {64, 8, (cuuint32_t)halves, by_group ? (cuuint32_t)P.box_rows / 8 : 1, 1};
    if (!encode(&qmap, f16, 3, a.q, qdims, qstr, qbox) || !encode(&kmap, f16, 5, a.k, kdims, kstr, kbox) ||
        !encode(&vmap, f16, 5, a.v, kdims, kstr, kbox))
        return cudaErrorInvalidValue;
    cudaError_t e;
    if (few)
        e = launch_paged_few(P, f16, grid, qmap, kmap, vmap, stream);
    else if (a.d == 64)
        e = f16 ? dispatch<1, 64>(P, two, grid, qmap, kmap, vmap, stream)
                : dispatch<0, 64>(P, two, grid, qmap, kmap, vmap, stream);
    else
        e = f16 ? dispatch<1, 128>(P, two, grid, qmap, kmap, vmap, stream)
                : dispatch<0, 128>(P, two, grid, qmap, kmap, vmap, stream);
    if (e != cudaSuccess) return e;
    if (P.whole_sel) return cudaSuccess;      // nothing is cut
    return two ? merge<4>(P, f16, grid, 256, stream) : merge<8>(P, f16, grid, 128, stream);
}

}  // namespace nsa
