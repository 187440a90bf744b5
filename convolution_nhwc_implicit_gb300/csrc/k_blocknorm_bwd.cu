// The gradient of the norms around a block (k_blocknorm.cu has the formulas).
#include "blocknorm.cuh"

namespace bn {

// The sums of the CTA's threads over the rows side by side (two or more):
// take(sum, channel, value) for the sums FIRST and on, each by one thread, in every
// call the same.
// ent: shared, NS x P pairs a thread; free on entry, free again on return.
template <int FIRST, int NS, int VEC, typename F>
__device__ __forceinline__ void combine(const Lane<VEC, 1> &l, int slots, float2 (&acc)[SUMS][4], float2 *ent, F &&take) {
    constexpr int P = 4;
    const int tpr = l.tpr, line = tpr < 32 ? tpr : 32;
    // rows of a part of a warp: first those of the warp, to every lane
    for (int o = line; o < 32; o *= 2)
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 &v = acc[FIRST + s][i];
                v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
                v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
            }
    const int rows = tpr < 32 ? blockDim.x / 32 : slots, wide = rows * tpr;
    const int me = tpr < 32 ? (threadIdx.x >> 5) * tpr + (threadIdx.x & 31) : threadIdx.x;
    __syncthreads();
    if ((threadIdx.x & 31) < line)
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < P; ++i) ent[(s * P + i) * wide + me] = acc[FIRST + s][i];
    __syncthreads();
    // one (sum, pair, thread of a row) at a time, those of a sum next to one another
    for (int k = threadIdx.x; k < NS * P * tpr; k += blockDim.x) {
        const int at = k / tpr, t = k - at * tpr;
        const float2 *e = ent + at * wide + t;
        float2 v = e[0];
        for (int r = 1; r < rows; ++r) v = add2(v, e[r * tpr]);
        Lane<VEC, 1> o = l;
        o.t = t;
        const int s = at / P, i = at - s * P;
        if (o.has(i, 0)) take(FIRST + s, o.chan(i, 0), v.x);
        if (o.has(i, 1)) take(FIRST + s, o.chan(i, 1), v.y);
    }
    __syncthreads();
}

// A sum's place in the workspace: of unit, or CTA, `at`.
__device__ __forceinline__ float *place(const BnArgs &a, int at, int s, int c) { return a.part + ((long long)at * SUMS + s) * a.Cp + c; }
// A unit that is a whole image gives its dgate at once and adds gate times its
// sums to the CTA's.
__device__ __forceinline__ void add_image(const BnArgs &a, int n, int cta, bool first, int s, int c, float v) {
    float *p = place(a, cta, s, c);
    const float gate = a.gate[(long long)n * a.C + c];
    *p = first ? gate * v : fmaf(gate, v, *p);
}
// A thread's channels of a row of fp32 values, in the widest vectors that they lie in.
// (own: a row of the workspace, whose rows lie on 16 bytes)
template <int VEC>
__device__ __forceinline__ void store(const Lane<VEC, 1> &l, float *row, const float2 (&v)[4], bool own = true) {
    if (VEC % 4 == 0 && (own || (reinterpret_cast<uintptr_t>(row) & 15) == 0)) {
#pragma unroll
        for (int i = 0; i < 4; i += 2)
            if (l.has(i, 0)) *reinterpret_cast<float4 *>(row + l.chan(i, 0)) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (l.has(i, 0)) row[l.chan(i, 0)] = v[i].x;
        if (l.has(i, 1)) row[l.chan(i, 1)] = v[i].y;
    }
}
// add_image and the gate's gradient of a whole image, by the threads that hold its
// sums of their channels; these start anew.
template <int VEC>
__device__ __forceinline__ void add_own_image(const Lane<VEC, 1> &l, const BnArgs &a, int n, int cta, bool first, float2 (&acc)[SUMS][4]) {
    float2 gate[4];
    l.params(gate, a.gate + (long long)n * a.C, 0.0f);
    if (a.dgate) {
        float2 scale[4], g1[4], b1[4];
        l.params(scale, a.scale, 1.0f);
        l.params(g1, a.g1, 1.0f);
        l.params(b1, a.b1, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) scale[i] = mul2(scale[i], fma2(g1[i], acc[SUM_A][i], mul2(b1[i], acc[SUM_B][i])));
        store(l, a.dgate + (long long)n * a.C, scale, false);
    }
#pragma unroll
    for (int s = 0; s < SUM_G2; ++s) {
        float2 sum[4];
        if (first)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.0f, 0.0f);
        else l.params(sum, place(a, cta, s, 0), 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sum[i] = fma2(gate[i], acc[s][i], sum[i]);
            acc[s][i] = make_float2(0.0f, 0.0f);
        }
        store(l, place(a, cta, s, 0), sum);
    }
}
// What the parameters' gradients of a channel need of the others, loaded ahead.
struct Others {
    float scale, g1, b1;
    __device__ __forceinline__ Others(const BnArgs &a, int c, bool on)
        : scale(on && a.scale ? a.scale[c] : 1.0f), g1(on && a.g1 ? a.g1[c] : 1.0f), b1(on && a.b1 ? a.b1[c] : 0.0f) {}
    // (A and B over an image)
    __device__ __forceinline__ float gate(float A, float B) const { return scale * (g1 * A + b1 * B); }
    // from the sums over all pixels, A and B times the gates
    __device__ __forceinline__ void put(const BnArgs &a, int c, float A, float B, float G2, float B2) const {
        if (a.dscale) a.dscale[c] = g1 * A + b1 * B;
        if (a.dg1) a.dg1[c] = scale * A;
        if (a.db1) a.db1[c] = scale * B;
        if (a.dg2) a.dg2[c] = G2;
        if (a.db2) a.db2[c] = B2;
    }
};

// The CTAs of a cluster, a unit each, join their sums: `mine` [SUMS][Cp] is the
// calling CTA's, which joins a share of the channels, a thread each (the last
// CTAs' shares may be empty).  What a channel needs besides is on its way while
// the CTAs wait for one another, which each of them does between its arrivals.
__device__ __forceinline__ void join_cluster(const BnArgs &a, const float *mine) {
    cluster_arrive();
    const int ranks = (int)gridDim.x, share = (a.C + ranks - 1) / ranks, c0 = (int)blockIdx.x * share, c1 = min(a.C, c0 + share);
    if (c0 >= c1) cluster_wait();
    for (int c = c0 + threadIdx.x; c - (int)threadIdx.x < c1; c += blockDim.x) {
        const bool on = c < c1, first = c == c0 + (int)threadIdx.x;
        const Others others(a, c, on);
        float gate[kCluster];
#pragma unroll
        for (int n = 0; n < kCluster; ++n) gate[n] = on && a.gate && n < a.N ? a.gate[(long long)n * a.C + c] : 1.0f;
        if (first) cluster_wait();
        if (!on) continue;
        const uint32_t at = tc::smem_u32(mine + c);
        float v[SUMS][kCluster];
#pragma unroll
        for (int r = 0; r < kCluster; ++r)
            if (r < ranks) {
                const uint32_t peer = tc::mapa_shared(at, r);
#pragma unroll
                for (int s = 0; s < SUMS; ++s)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[s][r]) : "r"(peer + s * a.Cp * 4) : "memory");
            }
        float A = 0.0f, B = 0.0f, G2 = 0.0f, B2 = 0.0f, ia = 0.0f, ib = 0.0f;
#pragma unroll
        for (int r = 0; r < kCluster; ++r)  // (S CTAs an image; without a gate, all of one)
            if (r < ranks) {
                ia += v[SUM_A][r];
                ib += v[SUM_B][r];
                G2 += v[SUM_G2][r];
                B2 += v[SUM_B2][r];
                if ((r + 1) % a.S == 0) {
                    const int n = r / a.S;
                    float k = gate[0];
#pragma unroll
                    for (int j = 1; j < kCluster; ++j) k = n == j ? gate[j] : k;
                    if (a.dgate) a.dgate[(long long)n * a.C + c] = others.gate(ia, ib);
                    A = fmaf(k, ia, A);
                    B = fmaf(k, ib, B);
                    ia = ib = 0.0f;
                }
            }
        others.put(a, c, A, B, G2, B2);
    }
    cluster_arrive();  // (no CTA ends while its sums may still be read)
    cluster_wait();
}

// Eight sums over a row that a cluster of two CTAs holds, half each.  A warp halves
// them over its lanes three times (a lane then holds one of them) and leaves them
// in both CTAs' shared memory, in one of two sets of entries in turn (as in
// RowSum); a lane then reads four of a warp's of each CTA.
struct PairSums {
    static constexpr int kWarps = kMostThreads / 32, kSet = 2 * kWarps * 2;
    float4 *buf;  // [2][CTA][warp][2]
    uint32_t peer;
    int rank, warps, flip;
    __device__ __forceinline__ PairSums(float4 *b, int rank_, int tpr)
        : buf(b), peer(tc::mapa_shared(tc::smem_u32(b), rank_ ^ 1)), rank(rank_), warps(tpr / 32), flip(0) {}
    __device__ static __forceinline__ float across(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
    __device__ static __forceinline__ float halved(bool hi, float a, float b, int o) { return (hi ? b : a) + across(hi ? a : b, o); }
    __device__ __forceinline__ void give(const float (&v)[8]) {
        const int lane = threadIdx.x & 31;
        const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = halved(h16, v[i], v[i + 4], 16);
        float f = halved(h4, halved(h8, a[0], a[2], 8), halved(h8, a[1], a[3], 8), 4);
        f += across(f, 2);
        f += across(f, 1);
        if ((lane & 3) == 0) {
            const int at = (flip + (rank * kWarps + (threadIdx.x >> 5)) * 2) * 4 + lane / 4;
            reinterpret_cast<float *>(buf)[at] = f;
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer + at * 4), "f"(f) : "memory");
        }
        cluster_arrive();
    }
    // (what lies between give and take hides a part of the way)
    __device__ __forceinline__ void take(float (&v)[8]) {
        const int lane = threadIdx.x & 31;
        const bool h16 = lane & 16, h8 = lane & 8;
        const float4 *e = buf + flip + lane;
        flip ^= kSet;
        cluster_wait();
        float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (lane < 2 * warps) {
            const float4 x = e[0], y = e[2 * kWarps];
            w = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        float f = halved(h8, halved(h16, w.x, w.z, 16), halved(h16, w.y, w.w, 16), 8);
        f += across(f, 4);
        f += across(f, 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(0xffffffffu, f, (i & 4 ? 1 : 0) | (i & 2 ? 16 : 0) | (i & 1 ? 8 : 0));
    }
};

// dx and df of the rows of a CTA's units, and the units' channel sums.  ALL: the
// block, dy and dz are given; what is then not asked for is formed all the same,
// which is fewer instructions than asking (8x80x80x256 bf16: 18.5 M warp
// instructions with the branches, 13.7 M without).  Normalised values are
// (v - m) r: as v r - m r, one instruction fewer a norm, they bore the rounding of
// m r, many times their own where the mean is far above the spread (8x80x80x256
// 31.6 us either way, 8x40x40x511 41.8 so and 42.8).  The statistics come through
// the ring too: read a row ahead they were what the warps waited for (37 us, 31.5
// so).  A pair of CTAs (ROW_PAIR) meets once a row, for the sums of both norms: a
// meeting of the cluster takes about half a microsecond (4096x8192 bf16 143 us with
// two, 106 with one, 98 with its sums written as vectors; floor 60).  Within a CTA
// one meeting for both gained less than its instructions cost up to 1024 channels
// and 4 % at 4096, and was not taken.
template <typename T, int VEC, int ROW, bool ALL, bool CUT>
__global__ void __launch_bounds__(kMostThreads) bn_bwd_kernel(const __grid_constant__ BnArgs a) {
    using R = Row<T, VEC, 1, CUT>;
    using Slot = typename R::Slot;
    constexpr int P = R::P, D = bwd_stages(), LINE = R::NV * R::step, STAGE = 4 * LINE;
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr bool PAIR = ROW == ROW_PAIR;
    __shared__ float4 meet[PAIR ? 2 * PairSums::kSet : 2 * kMeet];
    const int nt = blockDim.x;
    Slot *ring = R::ring(smem, D * 4);  // [D][x, f, dy, dz]
    const int rank = PAIR ? blockIdx.x & 1 : 0, cta = PAIR ? blockIdx.x >> 1 : blockIdx.x, ctas = PAIR ? gridDim.x >> 1 : gridDim.x;
    Lane<VEC, 1> l(a);
    if (PAIR) l.t += rank * R::NV * a.tpr;
    // statistics [warp][D][rows of a warp], copied by a lane of each row
    const int line = l.tpr < 32 ? l.tpr : 32, lane = threadIdx.x & 31;
    float4 *const seen = reinterpret_cast<float4 *>(smem + (size_t)D * 4 * R::NV * nt * sizeof(Slot)) +
                         (threadIdx.x >> 5) * (D * (32 / line)) + lane / line;
    const bool copies = lane % line == 0;
    float2 *const ent = reinterpret_cast<float2 *>(smem);  // after a unit's rows: the threads' sums
    // (fp32: with both ways of meeting, 36 bytes of a thread's registers are spilled,
    // and 8192x4096 takes 171 us for 135)
    RowSum<PAIR ? ROW_WARP : ROW, sizeof(T) == 2> sum(a.tpr, l.slot, meet);
    PairSums pair(meet, rank, a.tpr);
    const bool block = ALL || a.f, stream = ALL || a.dy, norm = ALL || a.dz;
    const float mean_post = a.post == CONV_NORM_LAYER ? -a.inv_c : 0.0f, mean_pre = a.pre == CONV_NORM_LAYER ? -a.inv_c : 0.0f;
    const long long sx = a.slots * a.px, sf = a.slots * a.pf, sdy = a.slots * a.pdy, sdz = a.slots * a.pdz;
    const long long s0 = a.slots * a.p0, s1 = a.slots * a.p1;
    pdl_trigger();
    pdl_wait();
    if (PAIR) cluster_arrive();
    float2 q[P], p[P], g2[P], acc[SUMS][P];
#pragma unroll
    for (int s = 0; s < SUMS; ++s)
#pragma unroll
        for (int i = 0; i < P; ++i) acc[s][i] = make_float2(0.0f, 0.0f);
    l.params(g2, a.g2, 1.0f);
    if (block && !a.gate) factors(l, a, 0, q, p);
    if (PAIR) cluster_wait();  // (the other CTA's shared memory is there)
    for (int unit = cta; unit < a.units; unit += ctas) {
        const int n = unit / a.S, k0 = unit - n * a.S;
        const int span = a.gate ? a.HW : a.rows;
        const int r0 = n * span + min(span, k0 * a.run), r1 = n * span + min(span, (k0 + 1) * a.run);
        int row = r0 + l.slot, asked = row;
        const T *x = static_cast<const T *>(a.x) + row * a.px + l.first(0), *f = static_cast<const T *>(a.f) + row * a.pf + l.first(0);
        const T *dy = static_cast<const T *>(a.dy) + row * a.pdy + l.first(0), *dz = static_cast<const T *>(a.dz) + row * a.pdz + l.first(0);
        T *dx = static_cast<T *>(a.o0) + row * a.p0 + l.first(0), *df = static_cast<T *>(a.o1) + row * a.p1 + l.first(0);
        unsigned ox = R::odd(x), of = R::odd(f), ody = R::odd(dy), odz = R::odd(dz);
        if (!a.full) R::template blank<D * 4>(l, ring);  // (the sums were there between units)
        const Slot *d = ring;
        Slot *to = ring;
        const float4 *sd = seen;
        float4 *sto = seen;
        __syncwarp();  // (every lane has read the last unit's statistics)
        // A row beyond the run counts as zeros.
        auto ask = [&](auto start) {  // (whether the map's first row may be it)
            constexpr bool START = decltype(start)::value;
            if (asked < r1) {
                if (copies) copy_async<16>(tc::smem_u32(sto), a.stats + asked);
                const bool late = CUT && START && asked == 0 && l.t == 0, bottom = CUT && asked == a.rows - 1;
                const int upto = bottom ? l.C - 1 : l.C;
                R::ask(l, x, to, upto, late);
                if (block) R::ask(l, f, to + LINE, upto, late);
                if (stream) R::ask(l, dy, to + 2 * LINE, upto, late);
                if (norm) R::ask(l, dz, to + 3 * LINE, upto, late);
                if (bottom && l.t == a.last_t && !(late && upto == 0)) {
                    const int at = a.last_v * a.tpr, slot = a.last_v * R::step;
                    R::ask_last(x + at, to + slot);
                    if (block) R::ask_last(f + at, to + LINE + slot);
                    if (stream) R::ask_last(dy + at, to + 2 * LINE + slot);
                    if (norm) R::ask_last(dz + at, to + 3 * LINE + slot);
                }
                if (late) {
                    R::ask_first(x, to, upto == 0);
                    if (block) R::ask_first(f, to + LINE, upto == 0);
                    if (stream) R::ask_first(dy, to + 2 * LINE, upto == 0);
                    if (norm) R::ask_first(dz, to + 3 * LINE, upto == 0);
                }
            } else {
                if (copies) *sto = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int m = 0; m < 4; ++m) R::zero(to + m * LINE);
            }
            copy_commit();
            asked += a.slots;
            x += sx;
            f += sf;
            dy += sdy;
            dz += sdz;
            const bool last = to == ring + (D - 1) * STAGE;
            to = last ? ring : to + STAGE;
            sto = last ? seen : sto + 32 / line;
        };
#pragma unroll
        for (int i = 0; i < D - 1; ++i) ask(std::true_type());
        if (block && a.gate) factors(l, a, n, q, p);
        for (int base = r0; base < r1; base += a.slots) {
            const bool on = row < r1;
            copy_wait<D - 2>();
            __syncwarp();
            const float4 st = *sd;
            float2 u[P], y[P], t[P];  // u^, y^, dY
            R::get(l, d, ox, y);
            if (block) {
                R::get(l, d + LINE, of, u);
                const float2 r = both(st.y), m = both(-st.x);
                if (ALL || a.b1)
#pragma unroll
                    for (int k = 0; k < P; ++k) y[k] = add2(y[k], p[k]);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    u[k] = mul2(add2(u[k], m), r);
                    y[k] = fma2(q[k], u[k], y[k]);
                }
            }
            if (stream) R::get(l, d + 2 * LINE, ody, t);
            else
#pragma unroll
                for (int k = 0; k < P; ++k) t[k] = make_float2(0.0f, 0.0f);
            float2 both_norms = make_float2(0.0f, 0.0f);  // PAIR: the sums of dY q and of dY q u^
            if constexpr (PAIR) {
                // One exchange: dY = T + m + my y^ of T = dy + r2 g2 dz, so that the sums of
                // dY q and of dY q u^ are made of T's, q's and y^ q's.  (They lose what T, m and
                // my y^ cancel, as the roundings of each dY do.)
                float2 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = make_float2(0.0f, 0.0f);
                if (norm) {
                    float2 e[P];
                    R::get(l, d + 3 * LINE, odz, e);
                    const float2 r = both(st.w), mean = both(-st.z);
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        acc[SUM_B2][k] = add2(acc[SUM_B2][k], e[k]);
                        y[k] = mul2(add2(y[k], mean), r);
                        acc[SUM_G2][k] = fma2(e[k], y[k], acc[SUM_G2][k]);
                        e[k] = mul2(e[k], g2[k]);
                        t[k] = fma2(e[k], r, t[k]);
                        w[0] = add2(w[0], e[k]);
                        w[1] = fma2(e[k], y[k], w[1]);
                    }
                } else
#pragma unroll
                    for (int k = 0; k < P; ++k) y[k] = make_float2(0.0f, 0.0f);
                if (block && a.post != CONV_NORM_NONE)
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        const float2 tq = mul2(t[k], q[k]), yq = mul2(y[k], q[k]);
                        w[2] = add2(w[2], tq);
                        w[3] = fma2(tq, u[k], w[3]);
                        w[4] = add2(w[4], q[k]);
                        w[5] = add2(w[5], yq);
                        w[6] = fma2(q[k], u[k], w[6]);
                        w[7] = fma2(yq, u[k], w[7]);
                    }
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = w[i].x + w[i].y;
                pair.give(v);
                ask(std::false_type());
                pair.take(v);
                // (without the second norm its statistics may be anything)
                const float my = norm ? -v[1] * a.inv_c * st.w : 0.0f, m = norm ? v[0] * mean_pre * st.w : 0.0f;
                both_norms = make_float2(fmaf(my, v[5], fmaf(m, v[4], v[2])), fmaf(my, v[7], fmaf(m, v[6], v[3])));
#pragma unroll
                for (int k = 0; k < P; ++k) t[k] = fma2(y[k], both(my), add2(t[k], both(m)));
            } else if (norm) {
                float2 e[P], w = make_float2(0.0f, 0.0f), v = w;
                R::get(l, d + 3 * LINE, odz, e);
                const float2 r = both(st.w), mean = both(-st.z);
                if (ALL || a.db2)
#pragma unroll
                    for (int k = 0; k < P; ++k) acc[SUM_B2][k] = add2(acc[SUM_B2][k], e[k]);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    y[k] = mul2(add2(y[k], mean), r);
                    acc[SUM_G2][k] = fma2(e[k], y[k], acc[SUM_G2][k]);
                    e[k] = mul2(e[k], g2[k]);
                    w = add2(w, e[k]);
                    v = fma2(e[k], y[k], v);
                }
                const float2 s = sum(w.x + w.y, v.x + v.y);
                const float2 my = both(-s.y * a.inv_c * st.w), m = both(s.x * mean_pre * st.w);
#pragma unroll
                for (int k = 0; k < P; ++k) t[k] = fma2(y[k], my, fma2(e[k], r, add2(t[k], m)));
            }
            const bool last = d == ring + (D - 1) * STAGE;
            d = last ? ring : d + STAGE;
            sd = last ? seen : sd + 32 / line;
            if (!PAIR) ask(std::false_type());
            if (on) R::put(l, dx, t);
            if (block) {
                // (what the mean's terms leave in a row beyond the run is 0: its sums are)
                if (ALL || a.want_b)
#pragma unroll
                    for (int k = 0; k < P; ++k) acc[SUM_B][k] = add2(acc[SUM_B][k], t[k]);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    acc[SUM_A][k] = fma2(t[k], u[k], acc[SUM_A][k]);
                    t[k] = mul2(t[k], q[k]);
                }
                if (a.post != CONV_NORM_NONE) {
                    float2 s = both_norms;
                    if (!PAIR) {
                        float2 w = make_float2(0.0f, 0.0f), v = w;
#pragma unroll
                        for (int k = 0; k < P; ++k) {
                            w = add2(w, t[k]);
                            v = fma2(t[k], u[k], v);
                        }
                        s = sum(w.x + w.y, v.x + v.y);
                    }
                    const float2 r = both(st.y), mu = both(-s.y * a.inv_c * st.y);
                    const float2 m = both(s.x * mean_post * st.y);
#pragma unroll
                    for (int k = 0; k < P; ++k) t[k] = fma2(u[k], mu, fma2(t[k], r, m));
                }
                if (on) R::put(l, df, t);
            }
            row += a.slots;
            dx += s0;
            df += s1;
            ox += (unsigned)sx;
            of += (unsigned)sf;
            ody += (unsigned)sdy;
            odz += (unsigned)sdz;
        }
        copy_wait<0>();
        // One row at a time: a thread holds its channels' sums of the CTA's rows, and
        // writes them as vectors (one value at a time, 32 bytes apart, took 8 us:
        // 152x4096 bf16 19.0 us and 10.4; 2048x1x1x1024 with a gate, which also went
        // through shared memory for its gradient, 50 and 26).
        if (PAIR || (ROW != ROW_PART && a.slots == 1 && !a.joined)) {
            if (!a.whole) {
#pragma unroll
                for (int s = 0; s < SUMS; ++s) store(l, place(a, unit, s, 0), acc[s]);
                continue;
            }
            add_own_image(l, a, n, cta, unit == cta, acc);
            if (unit + ctas >= a.units)
#pragma unroll
                for (int s = SUM_G2; s < SUMS; ++s) store(l, place(a, cta, s, 0), acc[s]);
            continue;
        }
        if (a.joined) break;  // (a CTA has one unit)
        if (a.whole) {
            const bool first = unit == (int)blockIdx.x;
            float *both_sums = reinterpret_cast<float *>(ent + 2 * P * nt);  // [A, B][C]: of a channel, two threads'
            combine<SUM_A, 2, VEC>(l, a.slots, acc, ent, [&](int s, int c, float v) {
                add_image(a, n, cta, first, s, c, v);
                if (a.dgate) both_sums[s * a.C + c] = v;
            });
            if (a.dgate) {
                __syncthreads();
                for (int c = threadIdx.x; c < a.C; c += nt) a.dgate[(long long)n * a.C + c] = Others(a, c, true).gate(both_sums[c], both_sums[a.C + c]);
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < P; ++i) acc[SUM_A][i] = acc[SUM_B][i] = make_float2(0.0f, 0.0f);
        } else combine<0, SUMS, VEC>(l, a.slots, acc, ent, [&](int s, int c, float v) { *place(a, unit, s, c) = v; });
    }
    if (PAIR || (ROW != ROW_PART && a.slots == 1 && !a.joined)) return;
    if (a.joined) {
        // (the CTA's sums after the threads')
        float *mine = reinterpret_cast<float *>(ent + (a.slots > 1 ? SUMS * P * nt : 0));
        if (ROW != ROW_PART && a.slots == 1) {
            __syncthreads();
#pragma unroll
            for (int s = 0; s < SUMS; ++s) store(l, mine + s * a.Cp, acc[s]);
        } else combine<0, SUMS, VEC>(l, a.slots, acc, ent, [&](int s, int c, float v) { mine[s * a.Cp + c] = v; });
        join_cluster(a, mine);
    } else if (a.whole)
        combine<SUM_G2, 2, VEC>(l, a.slots, acc, ent, [&](int s, int c, float v) { *place(a, blockIdx.x, s, c) = v; });
}

// Joins the units' sums: a CTA takes sixteen channels, four a thread, and 128
// units at a time.  Blocks y = 0 sum over all units; those above an image's
// units for its dgate, an image a warp.
constexpr int kJoin = 512, kJoinC = 16;
__device__ __forceinline__ void add4(float4 &s, const float4 &v, float k) {
    s.x = fmaf(k, v.x, s.x);
    s.y = fmaf(k, v.y, s.y);
    s.z = fmaf(k, v.z, s.z);
    s.w = fmaf(k, v.w, s.w);
}
__device__ __forceinline__ float4 sum8(float4 v) {  // over the lanes of one four of channels
#pragma unroll
    for (int o = 4; o < 32; o *= 2) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
        v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
    }
    return v;
}
__global__ void __launch_bounds__(kJoin) bn_join_kernel(const __grid_constant__ BnArgs a, int parts) {
    __shared__ float4 red[SUMS][kJoin / 32][kJoinC / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, four = lane & 3, group = lane >> 2;
    const int c = blockIdx.x * kJoinC + four * 4;  // (channels are padded to fours in the workspace)
    const bool on = c < a.C;
    pdl_trigger();
    pdl_wait();
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int at = blockIdx.x * kJoinC + (lane & 15);  // the first warp's channels, a lane each, twice
    const Others others(a, at, warp == 0 && at < a.C && blockIdx.y == 0);
    if (blockIdx.y > 0) {
        const int n = (blockIdx.y - 1) * (kJoin / 32) + warp;
        float4 A = zero, B = zero;
        if (n < a.N && on)
            for (int s = group; s < a.S; s += 8) {
                const float *u = a.part + ((long long)n * a.S + s) * SUMS * a.Cp + c;
                add4(A, *reinterpret_cast<const float4 *>(u + SUM_A * a.Cp), 1.0f);
                add4(B, *reinterpret_cast<const float4 *>(u + SUM_B * a.Cp), 1.0f);
            }
        A = sum8(A);
        B = sum8(B);
        if (n < a.N && group < 4 && c + group < a.C) {
            const int k = c + group;
            const float va = group == 0 ? A.x : (group == 1 ? A.y : (group == 2 ? A.z : A.w));
            const float vb = group == 0 ? B.x : (group == 1 ? B.y : (group == 2 ? B.z : B.w));
            a.dgate[(long long)n * a.C + k] = Others(a, k, true).gate(va, vb);
        }
        return;
    }
    float4 v[SUMS] = {zero, zero, zero, zero};
    const bool gated = a.gate && !a.whole;
    if (on)
        for (int u = warp * 8 + group; u < parts; u += kJoin / 4) {
            const float4 *one = reinterpret_cast<const float4 *>(a.part + (long long)u * SUMS * a.Cp + c);
            float4 w[SUMS];
#pragma unroll
            for (int s = 0; s < SUMS; ++s) w[s] = one[s * (a.Cp / 4)];
            if (gated) {
                const float *g = a.gate + (long long)(u / a.S) * a.C + c;
                const float4 k = make_float4(g[0], c + 1 < a.C ? g[1] : 0.0f, c + 2 < a.C ? g[2] : 0.0f, c + 3 < a.C ? g[3] : 0.0f);
#pragma unroll
                for (int s = 0; s < SUM_G2; ++s) w[s] = make_float4(k.x * w[s].x, k.y * w[s].y, k.z * w[s].z, k.w * w[s].w);
            }
#pragma unroll
            for (int s = 0; s < SUMS; ++s) add4(v[s], w[s], 1.0f);
        }
#pragma unroll
    for (int s = 0; s < SUMS; ++s) {
        v[s] = sum8(v[s]);
        if (group == 0) red[s][warp][four] = v[s];
    }
    __syncthreads();
    if (warp == 0) {
        float t[SUMS];
#pragma unroll
        for (int s = 0; s < SUMS; ++s) {
            t[s] = 0.0f;
            const float *r = reinterpret_cast<const float *>(red[s]) + (lane & 15);
            for (int w = lane >> 4; w < kJoin / 32; w += 2) t[s] += r[w * kJoinC];
            t[s] += __shfl_xor_sync(0xffffffffu, t[s], 16);
        }
        if (lane < 16 && at < a.C) others.put(a, at, t[SUM_A], t[SUM_B], t[SUM_G2], t[SUM_B2]);
    }
}

template <typename T, int VEC, bool CUT = false>
const void *pick(bool pair, int tpr, bool all) {
    if (pair) return all ? (const void *)&bn_bwd_kernel<T, VEC, ROW_PAIR, true, CUT> : (const void *)&bn_bwd_kernel<T, VEC, ROW_PAIR, false, CUT>;
    if (!all) return (const void *)&bn_bwd_kernel<T, VEC, ROW_ANY, false, CUT>;
    return tpr < 32 ? (const void *)&bn_bwd_kernel<T, VEC, ROW_PART, true, CUT>
                    : (tpr == 32 ? (const void *)&bn_bwd_kernel<T, VEC, ROW_WARP, true, CUT> : (const void *)&bn_bwd_kernel<T, VEC, ROW_WARPS, true, CUT>);
}
const void *pick_bwd(conv_dtype_t dt, int vec, bool cut, bool pair, int tpr, bool all) {
    using B = __nv_bfloat16;
    if (dt == CONV_F32) return vec == 4 ? pick<float, 4>(pair, tpr, all) : pick<float, 1>(pair, tpr, all);
    if (vec > 1) return vec == 8 ? pick<B, 8>(pair, tpr, all) : pick<B, 2>(pair, tpr, all);
    return cut ? pick<B, 1, true>(pair, tpr, all) : pick<B, 1>(pair, tpr, all);
}

cudaError_t launch_join(const BnArgs &a, int parts, cudaStream_t st) {
    BnArgs b = a;
    void *args[] = {&b, &parts};
    const bool images = a.dgate && !a.whole;
    const dim3 grid((unsigned)((a.C + kJoinC - 1) / kJoinC), 1 + (unsigned)(images ? (a.N + kJoin / 32 - 1) / (kJoin / 32) : 0));
    return conv_launch((const void *)&bn_join_kernel, grid, dim3(kJoin), args, 0, st);
}

}  // namespace bn
