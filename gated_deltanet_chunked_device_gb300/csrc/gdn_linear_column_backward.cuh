// gdn_linear_column_backward.cuh -- the backward pass of the gated linear
// recurrence with columns of channels streamed along the tokens, from the last
// token to the first (gdn_linear_column.cuh has the forward pass and the
// layout).
//
//     c_t = a_t g_t,  g_t = dy_t + c_{t+1}:   dx = b g, db = x g, da = h_{t-1} g
//
// The carry c is composed from the right as the forward pass composes the
// state from the left.  The states h are composed from the left again, inside
// a tile of 64 tokens only: the forward pass has saved the state at each
// tile's end (1/64 of fp32 states; recomputing them from the sequence's start
// would be another pass over x, a and b).  x, dy and b are read from shared
// memory twice, so that a run's registers are its gates, u = b x and the
// states that take u's place.
//
// 32768 x 4096: 312 us in bf16 with gates per channel (0.89 of a measured
// copy), 458 us with fp32 gates (0.95), 554 us in fp32 (1.0); with gates per
// head 224 us (0.54).  There nothing is full: 59 % of the issue slots, no pipe
// above 36 %, and 24 of the 152 SMs without a block.  A fifth of a warp's 960
// instructions a stage are the sums over a head's channels, which have a fixed
// order: over a thread's 4 channels, over a run's lanes by exchanges that halve
// the tokens a lane has sums of, and over the blocks of a head by a small
// kernel (9 us), in place of atomics whose order would change the result.
#pragma once

#include "gdn_linear_column.cuh"

namespace gdn {
namespace linear {

template <class X, class G, int kGates, bool kHasB, class Col>
struct BackwardShape {
    static constexpr int W = Col::kWidth, kTokens = Col::kTokens;
    using AX = StageArray<X, Col>;
    using AG = std::conditional_t<kGates == kOneHead, StageGates<G, Col>, StageArray<G, Col>>;
    // dy, a, x, b: the first two are what a pass that learns needs
    static constexpr int kLearnBytes = AX::kBytes + AG::kBytes;
    static constexpr int kStageBytes = 2 * AX::kBytes + (kHasB ? 2 : 1) * AG::kBytes;
    static constexpr int kDepth = kRingBytes / kStageBytes < 6 ? kRingBytes / kStageBytes : 6;
    struct Group {
        StageBounds<kTokens> bounds[3];
        alignas(16) float2 pairs[2][Col::kWarps][W];  // a warp's tokens: product of the gates, carry from zero
        alignas(16) float states[2][Col::kWarps][W];  // and the state from zero
    };
    struct Tables {
        Group groups[Col::kGroups];
        float hand[Col::kHands][W];   // the carry that enters a stage
        int32_t hand_reset[Col::kHands];
        Product product[Col::kSegments ? Col::kGroups * Col::kWarps : 1][W];  // of the gates of a warp's steps that learn
        uint64_t full[kDepth];
        uint64_t handed[Col::kHands];
        uint32_t ticket;
    };
    static constexpr int kSmem = kDepth * kStageBytes + static_cast<int>(sizeof(Tables));
    static_assert(kDepth >= 2, "the next stage comes while one is worked on");
    static_assert(kStageBytes % 128 == 0 && alignof(Tables) == 16, "boxes and tables lie aligned");
    static_assert(kSmem <= 227 * 1024, "shared memory of a block");
};

template <class X, class G, int kGates, bool kHasB, class Col>
__global__ void __launch_bounds__(Col::kThreads, 1)
    gdn_linear_column_backward_kernel(const LinearParams p, const Segments seg, const __grid_constant__ ColumnMaps maps) {
    using Shape = BackwardShape<X, G, kGates, kHasB, Col>;
    using AX = typename Shape::AX;
    using AG = typename Shape::AG;
    constexpr int W = Shape::W, kTokens = Shape::kTokens, kDepth = Shape::kDepth, kRuns = Col::kRuns, kLanesRow = Col::kLanesRow;
    constexpr int kColWarps = Col::kWarps, kWarpTokens = Col::kWarpTokens, kRun = Col::kRun, kGroups = Col::kGroups;
    constexpr int kHands = Col::kHands;
    constexpr int kTileWarps = kTile / kWarpTokens;  // warps whose tokens are a tile
    extern __shared__ __align__(1024) uint8_t ring[];
    typename Shape::Tables& sm = *reinterpret_cast<typename Shape::Tables*>(ring + kDepth * Shape::kStageBytes);
    const int group = threadIdx.x / (32 * kColWarps), warp = threadIdx.x / 32 % kColWarps, lane = threadIdx.x % 32;
    typename Shape::Group& gr = sm.groups[group];
    const bool leader = warp == 0 && lane == 0;  // of the group
    const int sub = lane / kLanesRow, l = lane % kLanesRow, run = warp * kRuns + sub, ch = lane % W;
    const ScanSpace& sp = seg.space;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kDepth; ++i) mbar_init(&sm.full[i], 1);
        for (int i = 0; i < kHands; ++i) mbar_init(&sm.handed[i], 1);
        fence_mbar_init();
        mbar_arrive(&sm.handed[0]);  // nothing is handed to stage 0: its place's first turn is over
        if (Col::kSegments) sm.ticket = atomicAdd(sp.ticket, 1u);
    }
    if (Col::kSegments) sm.product[threadIdx.x / 32][lane] = Product{1.f, 0};
    __syncthreads();
    const uint32_t ticket = Col::kSegments ? sm.ticket : blockIdx.x;
    const int64_t part = Col::kSegments ? ticket / sp.blocks : 0;  // segments are counted from the right
    const uint32_t blk = Col::kSegments ? ticket % sp.blocks : ticket;
    const int c0 = static_cast<int>(blk) * W, cols = min(W, p.C - c0);
    // stages of the whole axis are counted from the left; this segment has [left, right)
    const int64_t all = max(static_cast<int64_t>(1), (p.T + kTokens - 1) / kTokens);
    const int64_t right = part == 0 ? all : all - seg.first - (part - 1) * seg.stages;
    const int64_t left = !Col::kSegments || part == sp.nt - 1 ? 0 : all - seg.first - part * seg.stages;
    const int stages = static_cast<int>(right - left);
    const bool twice = Col::kSegments && part > 0;
    const int steps = p.T == 0 ? 0 : twice ? 2 * stages : stages;
    const bool on = l * 4 < cols;
    const int head = c0 / p.D;

    auto stage_start = [&](int q) { return (right - 1 - (q < stages ? q : q - stages)) * kTokens; };
    auto fetch = [&](int q) {  // one thread
        if (q >= steps) return;
        uint8_t* stage = ring + q % kDepth * Shape::kStageBytes;
        uint64_t* bar = &sm.full[q % kDepth];
        const int64_t t0 = stage_start(q);
        const int at = kGates == kOneHead ? head : c0;
        const bool learn = twice && q < stages;
        mbar_arrive_expect_tx(bar, learn ? Shape::kLearnBytes : Shape::kStageBytes);
        AX::fetch(stage, &maps.dy, bar, c0, t0);
        AG::fetch(stage + AX::kBytes, &maps.a, bar, at, t0);
        if (learn) return;
        AX::fetch(stage + Shape::kLearnBytes, &maps.x, bar, c0, t0);
        if constexpr (kHasB) AG::fetch(stage + Shape::kLearnBytes + AX::kBytes, &maps.b, bar, at, t0);
    };
    Window win{0, 0};  // from the first entry past the tokens to come down
    auto bounds = [&](int q) {
        if (q >= max(steps, 1)) return;  // without tokens, the empty sequences
        const int64_t t0 = stage_start(q), t1 = min(t0 + kTokens, p.T);
        if (q < kGroups || (q >= stages && q < stages + kGroups))
            win.load(p, first_entry(p, static_cast<int64_t>(p.N) + 1, t1 + 1, lane), -1, lane);
        StageBounds<kTokens>& b = gr.bounds[q / kGroups % 3];
        if (t1 == t0 + kTokens && !__any_sync(0xffffffffu, win.c >= t0 && win.c <= t1) && __any_sync(0xffffffffu, win.c < t0)) {
            no_bounds(b, lane);  // most stages
            return;
        }
        const bool write = q >= steps - stages, last = t1 == p.T;
        auto empty = [&](int64_t i) {  // an empty sequence hands the gradient of its final state on
            if (!write || !p.d_initial || lane * 4 >= cols) return;
            const int64_t off = i * p.C + c0 + lane * 4;
            *reinterpret_cast<float4*>(p.d_initial + off) =
                p.d_final ? *reinterpret_cast<const float4*>(p.d_final + off) : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        if (__shfl_sync(0xffffffffu, win.c, 31) < t0) {  // the window holds all of the stage's entries
            clear_bounds<kTokens>(b, lane);
            const int64_t prev = __shfl_down_sync(0xffffffffu, win.c, 1), next = __shfl_up_sync(0xffffffffu, win.c, 1);
            const bool gap = lane > 0 && mark_entry<kTokens>(p, win.first - lane, win.c, prev, next, t0, t1, last, b, [&](bool start, int64_t i) {
                if (start && p.initial_state)
                    prefetch_l2(static_cast<const uint8_t*>(p.initial_state) + (i * p.state_stride + c0) * dtype_bytes(p.state_dt));
                if (!start && p.d_final) prefetch_l2(p.d_final + i * p.C + c0);
            });
            for (uint32_t m = __ballot_sync(0xffffffffu, gap); m; m &= m - 1) empty(win.first - (__ffs(m) - 1));
            sum_up_bounds<kTokens, kWarpTokens>(t0, t1, lane, b);
            win.load(p, win.first - __popc(__ballot_sync(0xffffffffu, win.c > t0)) + 1, -1, lane);
        } else {
            const int64_t n = static_cast<int64_t>(p.N) + 1;
            fill_bounds<kTokens, kWarpTokens>(p, first_entry(p, n, t0, lane), t0, t1, last, lane, b, empty);
            win.load(p, first_entry(p, n, t0 + 1, lane), -1, lane);
        }
    };
    // The state that enters this warp's tile (of channel `ch`), from the forward pass: one step ahead.
    float saved = 0.f;
    auto fetch_saved = [&](int q) {
        saved = 0.f;
        if (q >= steps || q < steps - stages || ch >= cols) return;
        const int64_t tile = stage_start(q) / kTile + warp / kTileWarps;
        if (tile > 0 && tile * kTile < p.T) saved = p.tile_states[(tile - 1) * p.C + c0 + ch];
    };

    // A stage's place in the ring is free when its group is done with it, which the group's next step shows: a place is
    // fetched kGroups stages late.
    constexpr int kAhead = kDepth - kGroups;
    static_assert(kAhead >= kGroups, "every group has its next stage on the way");
    if (threadIdx.x == 0)
        for (int q = 0; q < kAhead; ++q) fetch(q);
    if (warp == kColWarps - 1) bounds(group);
    if (group == 0 && warp == 0 && blk == 0) check_bounds(p, part, sp.nt, lane);
    fetch_saved(group);
    __syncthreads();
    bool ok = true;  // until a wait runs out; then what this thread adds to the results is NaN
    auto wait = [&](uint64_t* bar, uint32_t parity, long long cycles) {
        if (!ok || mbar_wait(bar, parity, cycles)) return;
        ok = false;
        report(p.status, GDN_DEVICE_ERR_TIMEOUT);
    };
    float own = 0.f;
    bool own_reset = false;
    auto wait_hand = [&](int q) { wait(&sm.handed[q % kHands], (q / kHands) & 1, hand_wait(sp.wait_cycles)); };
    const int pieces = kGates == kOneHead ? p.D / W : 1, piece = kGates == kOneHead ? c0 % p.D / W : 0;
    for (int q = group; q < steps; q += kGroups) {
        const StageBounds<kTokens>& bd = gr.bounds[q / kGroups % 3];
        const bool learn = twice && q < stages;
        const int64_t t = stage_start(q) + run * kRun;
        uint8_t *stage = ring + q % kDepth * Shape::kStageBytes, *sx = stage + Shape::kLearnBytes;
        const uint8_t *sa = stage + AX::kBytes, *sb = sx + AX::kBytes;
        using Gate = std::conditional_t<kGates == kPerChannel, Quad, float>;
        Gate a[kRun], A, exA, rxA;
        Quad u[kRun], B = all4(0.f), E, exB, rxE;
        constexpr int kHeld = kGates == kOneHead ? (kRun + kLanesRow - 1) / kLanesRow : 1;
        float ha[kHeld], hb[kHeld];
        uint32_t starts = 0, ends = 0;
        int n = kRun;
        bool plain = true, started = false, ended = false;  // whether a sequence starts in the runs before, ends in those after
        uint32_t any_start = 0, any_end = 0;
        auto initial = [&](int k) {
            if (!p.initial_state || !on) return all4(0.f);
            return quad(state_quad_load(p.initial_state, bd.start_seq[run * kRun + k] * p.state_stride + c0 + l * 4, p.state_dt));
        };
        auto final_gradient = [&](int k) {
            if (!p.d_final || !on) return all4(0.f);
            return quad(state_quad_load(p.d_final, static_cast<int64_t>(bd.end_seq[run * kRun + k]) * p.C + c0 + l * 4, GDN_DTYPE_F32));
        };
        // gates of one head: lane l of a run holds the run's token l
        auto shared_gate = [&](const float(&held)[kHeld], int k) {
            return __shfl_sync(0xffffffffu, held[k / kLanesRow], sub * kLanesRow + k % kLanesRow);
        };
        if (warp == kColWarps - 1) bounds(q + kGroups);
        plain = (bd.plain >> warp) & 1;
        wait(&sm.full[q % kDepth], (q / kDepth) & 1, copy_wait(sp.wait_cycles));
        if (!ok) {
            AX::spoil(stage, run, l);
            if (!learn) AX::spoil(sx, run, l);
        }
        if constexpr (kGates == kOneHead) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int tok = run * kRun + min(i * kLanesRow + l, kRun - 1);
                ha[i] = AG::get(sa, tok, head);
                if (kHasB && !learn) hb[i] = AG::get(sb, tok, head);
            }
        }
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            if constexpr (kGates == kOneHead)
                a[k] = shared_gate(ha, k);
            else
                a[k] = widen(AG::get(sa, run, k, l));
        }
        if (!learn) {
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                u[k] = widen(AX::get(sx, run, k, l));
                if constexpr (kHasB) {
                    if constexpr (kGates == kOneHead)
                        u[k] = mul(shared_gate(hb, k), u[k]);
                    else
                        u[k] = mul(u[k], widen(AG::get(sb, run, k, l)));
                }
            }
        }
        set_gate(A, 1.f);
        E = all4(0.f);
        if (!plain) {
            n = static_cast<int>(min(static_cast<int64_t>(kRun), max(static_cast<int64_t>(0), p.T - t)));
#pragma unroll
            for (int k = 0; k < kRun; ++k)  // past the end, a carry goes through
                if (k >= n) set_gate(a[k], 1.f);
            starts = run_bits<kRun>(bd.starts, run);
            ends = run_bits<kRun>(bd.ends, run);
            any_start = any_run_bits<kRun, kRuns>(bd.starts, warp);
            any_end = any_run_bits<kRun, kRuns>(bd.ends, warp);
        }
        // `whole`: all of the warp's tokens are there, with neither a start nor an end: code without a branch.
        auto compose = [&](auto whole) {
            constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
            for (int k = kRun - 1; k >= 0; --k) {
                if (!kWhole && ((any_end >> k) & 1) && ((ends >> k) & 1)) E = final_gradient(k);
                E = mul(a[k], add(widen(AX::get(stage, run, k, l)), E));
                A = mul(A, a[k]);
            }
            if (!learn)
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    if (!kWhole && ((any_start >> k) & 1) && ((starts >> k) & 1)) B = initial(k);
                    B = fma(a[k], B, u[k]);
                }
        };
        if (plain)
            compose(std::true_type{});
        else
            compose(std::false_type{});
        // over the warp's runs: the carry from the right, the state from the left
        const uint32_t rs = (bd.warps_start >> warp) & 1 ? runs_with<kRun, kRuns>(bd.starts, warp) : 0;
        const uint32_t re = (bd.warps_end >> warp) & 1 ? runs_with<kRun, kRuns>(bd.ends, warp) : 0;
        Gate RA = A;
#pragma unroll
        for (int o = 1; o < kRuns; o <<= 1) {
            const bool mine = (re >> sub) & ((1u << o) - 1u);
            const Gate oa = shift_down(RA, o * kLanesRow);
            const Quad oe = shift_down(E, o * kLanesRow);
            if (sub + o < kRuns) {
                E = pick(mine, E, fma(RA, oe, E));
                RA = mul(RA, oa);
            }
        }
        rxA = shift_down(RA, kLanesRow);
        rxE = shift_down(E, kLanesRow);
        if (sub == kRuns - 1) {
            set_gate(rxA, 1.f);
            rxE = all4(0.f);
        }
        ended = (re >> (sub + 1)) != 0;
        if (!learn) {
#pragma unroll
            for (int o = 1; o < kRuns; o <<= 1) {
                const bool mine = (rs >> max(0, sub - o + 1)) & ((1u << o) - 1u);
                const Gate oa = shift_up(A, o * kLanesRow);
                const Quad ob = shift_up(B, o * kLanesRow);
                if (sub >= o) {
                    B = pick(mine, B, fma(A, ob, B));
                    A = mul(A, oa);
                }
            }
            exA = shift_up(A, kLanesRow);
            exB = shift_up(B, kLanesRow);
            if (sub == 0) {
                set_gate(exA, 1.f);
                exB = all4(0.f);
            }
            started = (rs & ((1u << sub) - 1u)) != 0;
        }
        // the warp's: the product and the carry are the first run's
        if (sub == 0) {
            float4* o = reinterpret_cast<float4*>(&gr.pairs[q / kGroups & 1][warp][l * 4]);
            const Quad g = of_channels(RA);
            o[0] = make_float4(g.lo.x, E.lo.x, g.lo.y, E.lo.y);
            o[1] = make_float4(g.hi.x, E.hi.x, g.hi.y, E.hi.y);
        }
        // the state is the last run's
        if (kTileWarps > 1 && !learn && sub == kRuns - 1) *reinterpret_cast<float4*>(&gr.states[q / kGroups & 1][warp][l * 4]) = flat(B);
        if (learn) {
            __syncwarp();
            Product& mine = sm.product[threadIdx.x / 32][lane];
            mine = times(mine, gr.pairs[q / kGroups & 1][warp][lane].x);
        }
        // The group's one barrier of a step.  Past it: every warp's pair is there, nobody of the group reads its stage before
        // any more (its place in the ring is free), and the bounds of the group's next stage are known.
        named_bar_sync(1 + group, 32 * kColWarps);
        if (leader && ok) fetch(q + kAhead);
        float2 ae[kColWarps];
#pragma unroll
        for (int w = 0; w < kColWarps; ++w) ae[w] = gr.pairs[q / kGroups & 1][w][ch];
        // the state at the tile's start, through the tile's warps before this one
        float enter_h = saved;
#pragma unroll
        for (int w = 0; w < kTileWarps - 1; ++w) {
            const int v = warp / kTileWarps * kTileWarps + w;
            if (v >= warp) break;
            const float b = gr.states[q / kGroups & 1][v][ch];
            enter_h = (bd.warps_start >> v) & 1 ? b : fmaf(gr.pairs[q / kGroups & 1][v][ch].x, enter_h, b);
        }
        fetch_saved(q + kGroups);
        // What the stage to the right hands on: the carry (in steps that learn, from zero).
        const uint32_t resets = bd.warps_end;
        // (One group keeps it itself.)
        float carry = own;
        if (kGroups > 1 && q > 0) {
            wait_hand(q);
            carry = ok ? sm.hand[q % kHands][ch] : nanf("");
        }
        float enter_c = carry;
#pragma unroll
        for (int w = kColWarps - 1; w >= 0; --w) {
            if (w == warp) enter_c = carry;
            carry = fmaf(ae[w].x, carry, ae[w].y);
            if (resets != 0 && ((resets >> w) & 1)) carry = ae[w].y;
        }
        own = carry;
        own_reset |= resets != 0;
        if (warp == 0 && (kGroups > 1 || Col::kSegments)) {
            const bool reset = kGroups == 1 ? own_reset : resets != 0 || (learn && q > 0 && sm.hand_reset[q % kHands] != 0);
            const int c = c0 + lane;
            uint32_t* flags = sp.flags + static_cast<int64_t>(blk) * sp.nt;
            if (learn && q == stages - 1) {  // the segment's pair goes on, the carry that enters it comes
                const bool lastpart = part == sp.nt - 1;
                Product whole{1.f, 0};
                for (int i = 0; i < kGroups * kColWarps; ++i) whole = times(whole, sm.product[i][lane]);
                whole = folded(whole);
                if (!lastpart) {
                    if (lane < cols) {
                        if (reset) {
                            sp.known[part * p.C + c] = carry;
                        } else {
                            sp.pairs[part * p.C + c] = make_float2(whole.m, carry);
                            sp.exponents[part * p.C + c] = whole.e;
                        }
                    }
                    const bool scaled = __any_sync(0xffffffffu, whole.e != 0);
                    publish(flags + part, reset ? kKnown : scaled ? kScaledPair : kPair, lane);
                }
                const float v = look_back<true>(p, sp, flags, part, lane < cols ? c : p.C, lane, [](int64_t k) { return k; });
                if (!lastpart && !reset) {
                    if (lane < cols) sp.known[part * p.C + c] = pass_on(whole, v, carry);
                    publish(flags + part, kKnown, lane);
                }
                carry = v;
            } else if (Col::kSegments && part == 0 && q == steps - 1) {  // the first segment's carry
                if (lane < cols) sp.known[c] = carry;
                publish(flags, kKnown, lane);
            }
            if (lane < W) sm.hand[(q + 1) % kHands][lane] = carry;
            if constexpr (kGroups > 1) {
                if (lane == 0) sm.hand_reset[(q + 1) % kHands] = reset;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.handed[(q + 1) % kHands]);
            }
        }
        if (kGroups == 1 && learn && q == stages - 1) {
            named_bar_sync(1, 32 * kColWarps);
            own = sm.hand[(q + 1) % kHands][ch];
        }
        if (learn) continue;
        auto spread = [&](float v) {
            return Quad{{__shfl_sync(0xffffffffu, v, l * 4), __shfl_sync(0xffffffffu, v, l * 4 + 1)},
                        {__shfl_sync(0xffffffffu, v, l * 4 + 2), __shfl_sync(0xffffffffu, v, l * 4 + 3)}};
        };
        Quad h = pick(started, exB, fma(exA, spread(enter_h), exB));
        Quad c = pick(ended, rxE, fma(rxA, spread(enter_c), rxE));
        float sums[kGates == kOneHead ? kRun : 1][2];
        // The tokens once more.
        auto tokens = [&](auto whole) {
            constexpr bool kWhole = decltype(whole)::value;
            // States before each, from the left; they take u's place.
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                if (!kWhole && ((any_start >> k) & 1) && ((starts >> k) & 1)) h = initial(k);
                const Quad v = h;
                if (k < kRun - 1) h = fma(a[k], h, u[k]);
                u[k] = v;
            }
            // Gradients, from the right.
            X* dx = static_cast<X*>(p.dx) + (t + kRun - 1) * p.dx_stride + c0 + l * 4;
            [[maybe_unused]] G* da = static_cast<G*>(p.da) + (kGates == kOneHead ? 0 : (t + kRun - 1) * p.da_stride + c0 + l * 4);
            [[maybe_unused]] G* db = kHasB ? static_cast<G*>(p.db) + (kGates == kOneHead ? 0 : (t + kRun - 1) * p.db_stride + c0 + l * 4) : nullptr;
#pragma unroll
            for (int k = kRun - 1; k >= 0; --k) {
                if (!kWhole && ((any_end >> k) & 1) && ((ends >> k) & 1)) c = final_gradient(k);
                const Quad g = add(widen(AX::get(stage, run, k, l)), c);
                const Quad va = mul(g, u[k]), vb = mul(g, widen(AX::get(sx, run, k, l)));
                Quad vx = g;
                if constexpr (kHasB) {
                    if constexpr (kGates == kOneHead)
                        vx = mul(shared_gate(hb, k), g);
                    else
                        vx = mul(g, widen(AG::get(sb, run, k, l)));
                }
                c = mul(a[k], g);
                if ((kWhole || k < n) && on) {
                    store_stream(reinterpret_cast<Pack<X>*>(dx), narrow(vx, X{}));
                    if constexpr (kGates == kPerChannel) {
                        store_stream(reinterpret_cast<Pack<G>*>(da), narrow(va, G{}));
                        if constexpr (kHasB) store_stream(reinterpret_cast<Pack<G>*>(db), narrow(vb, G{}));
                    }
                }
                if (!kWhole && ((any_start >> k) & 1) && ((starts >> k) & 1) && on && p.d_initial)
                    *reinterpret_cast<float4*>(p.d_initial + static_cast<int64_t>(bd.start_seq[run * kRun + k]) * p.C + c0 + l * 4) = flat(c);
                dx -= p.dx_stride;
                if constexpr (kGates == kPerChannel) {
                    da -= p.da_stride;
                    if constexpr (kHasB) db -= p.db_stride;
                } else {
                    const float2 sa = add2(va.lo, va.hi), sb2 = add2(vb.lo, vb.hi);
                    sums[k][0] = sa.x + sa.y;
                    sums[k][1] = sb2.x + sb2.y;
                }
            }
        };
        if (plain)
            tokens(std::true_type{});
        else
            tokens(std::false_type{});
        if constexpr (kGates == kOneHead) {
            // Over the run's lanes: each exchange halves the tokens that a lane has sums of, until it has one (kRun / lanes).
            static_assert(kRun % kLanesRow == 0, "every lane ends with tokens of its own");
#pragma unroll
            for (int o = kLanesRow / 2, m = kRun; o > 0; o >>= 1) {
                m /= 2;
                const bool up = (l & o) != 0;
#pragma unroll
                for (int i = 0; i < m; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float keep = up ? sums[i + m][j] : sums[i][j], give = up ? sums[i][j] : sums[i + m][j];
                        sums[i][j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
            }
            constexpr int kMine = kRun / kLanesRow;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int k = l * kMine + i;
                if (k >= n) continue;
                const int64_t tk = t + k;
                if (pieces == 1) {
                    from_f32(sums[i][0], static_cast<G*>(p.da)[tk * p.da_stride + head]);
                    if constexpr (kHasB) from_f32(sums[i][1], static_cast<G*>(p.db)[tk * p.db_stride + head]);
                } else {
                    reinterpret_cast<float2*>(p.scratch)[(tk * p.H + head) * pieces + piece] = make_float2(sums[i][0], sums[i][1]);
                }
            }
        }
    }
    if (leader && !ok) drain(sm.full, sp.wait_cycles);
}

template <class X, class G, int kGates, bool kHasB, class Col>
cudaError_t launch_column_backward(const LinearParams& p, const Segments& seg, cudaStream_t stream) {
    using Shape = BackwardShape<X, G, kGates, kHasB, Col>;
    ColumnMaps maps{};
    if (p.T > 0) {
        const int64_t row = kGates == kOneHead ? p.H : p.C;
        const int width = kGates == kOneHead ? 16 / static_cast<int>(sizeof(G)) : Shape::W;
        bool ok = encode_rows(&maps.x, p.x, p.x_dt, p.x_stride, p.C, p.T, Shape::W, Shape::AX::kBox) &&
                  encode_rows(&maps.dy, p.dy, p.x_dt, p.dy_stride, p.C, p.T, Shape::W, Shape::AX::kBox) &&
                  encode_rows(&maps.a, p.a, p.gate_dt, p.a_stride, row, p.T, width, Shape::AG::kBox);
        if (kHasB) ok = ok && encode_rows(&maps.b, p.b, p.gate_dt, p.b_stride, row, p.T, width, Shape::AG::kBox);
        if (!ok) return cudaErrorInvalidValue;
    }
    auto kernel = gdn_linear_column_backward_kernel<X, G, kGates, kHasB, Col>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(seg.space.nt * seg.space.blocks), Col::kThreads, Shape::kSmem, stream>>>(p, seg, maps);
    if (kGates == kOneHead && p.D > Shape::W && p.T > 0)
        gdn_linear_join_kernel<G><<<static_cast<unsigned>((p.T * p.H + 255) / 256), 256, 0, stream>>>(p, p.D / Shape::W);
    return cudaGetLastError();
}

// Tokens of a run: 8, or 4 where gates per channel are fp32 and two stages of 8 would fill the ring.
template <class G, int kGates>
constexpr int backward_run() {
    return kGates == kPerChannel && sizeof(G) == 4 ? 4 : 8;
}

// Groups of 8 warps: two, where 128 registers a thread hold a run (of 8 tokens with gates per channel they do not), and the
// ring four stages (fp32 throughout: fewer).
template <class X, class G, int kGates>
constexpr int backward_groups() {
    return sizeof(X) == 4 || (kGates == kPerChannel && sizeof(G) == 2) ? 1 : 2;
}

template <class X, class G, int kGates>
cudaError_t column_backward_gates(const LinearParams& p, const Segments& seg, int width, cudaStream_t stream) {
    constexpr int R = backward_run<G, kGates>(), NG = backward_groups<X, G, kGates>();
    if (seg.space.nt > 1)
        return p.b ? launch_column_backward<X, G, kGates, true, Column<32, 8, R, NG, true>>(p, seg, stream)
                   : launch_column_backward<X, G, kGates, false, Column<32, 8, R, NG, true>>(p, seg, stream);
    if (width == 32)
        return p.b ? launch_column_backward<X, G, kGates, true, Column<32, 8, R, NG>>(p, seg, stream)
                   : launch_column_backward<X, G, kGates, false, Column<32, 8, R, NG>>(p, seg, stream);
    return p.b ? launch_column_backward<X, G, kGates, true, Column<16, 8, R, NG>>(p, seg, stream)
               : launch_column_backward<X, G, kGates, false, Column<16, 8, R, NG>>(p, seg, stream);
}

template <class X, class G>
cudaError_t column_backward_typed(const LinearParams& p, const Segments& seg, int width, cudaStream_t stream) {
    if (p.gate_div == 1) return column_backward_gates<X, G, kPerChannel>(p, seg, width, stream);
    return column_backward_gates<X, G, kOneHead>(p, seg, width, stream);
}

}  // namespace linear
}  // namespace gdn
