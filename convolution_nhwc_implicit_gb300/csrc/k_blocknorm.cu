// The norms before and after a block, fused with the block's gate, its residual
// scale and the residual add, over NHWC maps: forward and gradient.
//
// With x the residual stream, f the block's output, each pixel a row of C
// channels, and norms of kind layer (mean and deviation), rms (m = 0) or none
// (m = 0, r = 1):
//   u^ = (f - m1) r1        u = g1 u^ + b1
//   y  = x + scale[c] gate[n,c] u
//   y^ = (y - m2) r2        z = g2 y^ + b2
// and, with dy and dz,
//   e  = g2 dz              dY = dy + r2 (e - [layer] mean e - y^ mean(e y^))
//   v  = scale gate g1 dY   df = r1 (v - [layer] mean v - u^ mean(v u^))
//   dx = dY
//   dg2 = sum dz y^         db2 = sum dz
//   A[n,c] = sum_p dY u^    B[n,c] = sum_p dY
//   dgate = scale (g1 A + b1 B)          dscale = sum_n gate (g1 A + b1 B)
//   dg1 = sum_n scale gate A             db1 = sum_n scale gate B
// The gradient forms y again of x and f, which is as many bytes as reading y
// and spares its rounding.  About 20 operations an element forward and 45
// backward against 8 to 24 bytes moved: memory bounds it.
//
// A thread holds 8 K channels of a row (K = 2 where rows are long, or many and a
// warp's) and, in the gradient, the channels' sums over its rows; a row is shared
// by as many threads as that takes: lanes of a warp, or whole warps that meet in
// shared memory.  A CTA takes several rows side by side and a run of sets of them.
// Rows are copied ahead into a ring of shared memory (cp.async), each thread its
// own values, so that nothing waits for another thread but the sums over a row.
// All statistics and sums are fp32, in a fixed order: results do not change from
// run to run.  (A thread adds its rows' terms of a sum over pixels one after
// another: all rows of 4096 channels over 152 CTAs, of 16 channels over 256 times
// as many.)
//
// Measured on a GB300 by graph replay over changing inputs, of HBM's 6.7 TB/s:
// 8x80x80x256 bf16, both norms rms and a gate, 19.8 us forward (105 MB, 15.8 us of
// them; two layer norms 20.2) and 31.8 for the gradient (157 MB, 23.5);
// 8192x8192 bf16 91.9 (537 MB, 80.1); 16x160x160x128 fp32 139 and 200 (839 and
// 1258 MB, 125 and 188).  What a launch and a run's start and end take, about 5 us
// of the gradient, is most of the rest; the arithmetic keeps 33 to 58 % of the
// issue slots busy.  Instructions were what bounded it at first: two rows at a time, sums
// that share their exchanges, instances without branches on what is absent and
// addresses that advance took a third to a half of them out.
#include <math.h>
#include <stdio.h>

#include <new>

#include "blocknorm.cuh"

using namespace bn;

namespace {

// y and z of a run of rows, RB at a time.  With RB = 1 and one row of 8 channels
// a thread the rows that a CTA takes of a gated map may be of several images;
// otherwise a run is of one.  ALL: f, y and z are given.
template <typename T, int VEC, int K, int RB, int ROW, bool ALL, bool CUT>
__global__ void __launch_bounds__(kMostThreads) bn_fwd_kernel(const __grid_constant__ BnArgs a) {
    using R = Row<T, VEC, K, CUT>;
    using Slot = typename R::Slot;
    constexpr int P = R::P, D = fwd_stages(R::kElement, K), LINE = R::NV * R::step, STAGE = 2 * RB * LINE;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float4 meet[2 * kMeet];
    Slot *ring = R::ring(smem, D * 2 * RB);  // [D][x, f][RB]
    const Lane<VEC, K> l(a);
    RowSum<ROW> sum(a.tpr, l.slot, meet);
    const int n = RB > 1 ? blockIdx.x / a.S : 0, s0 = RB > 1 ? blockIdx.x - n * a.S : blockIdx.x;
    const int span = RB > 1 && a.S < a.units ? a.HW : a.rows;
    const int r0 = n * span + s0 * a.run, r1 = n * span + min(span, (s0 + 1) * a.run);
    int row = r0 + l.slot, asked = row;
    const bool block = ALL || a.f, norm = ALL || a.o1;
    const T *x = static_cast<const T *>(a.x) + row * a.px + l.first(0), *f = static_cast<const T *>(a.f) + row * a.pf + l.first(0);
    T *y = static_cast<T *>(a.o0) + row * a.p0 + l.first(0), *z = static_cast<T *>(a.o1) + row * a.p1 + l.first(0);
    const long long sx = a.slots * a.px, sf = a.slots * a.pf, sy = a.slots * a.p0, sz = a.slots * a.p1;
    // (of the rows at hand, and how they change from a row of the slot to its next)
    unsigned ox = R::odd(x), of = R::odd(f);
    const unsigned nx = sx & 1, nf = sf & 1;
    pdl_trigger();
    if (!a.full) R::template blank<D * 2 * RB>(l, ring);
    pdl_wait();
    const Slot *d = ring;
    Slot *to = ring;
    auto ask = [&](auto start) {  // (whether the map's first row may be among them)
        constexpr bool START = decltype(start)::value;
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            if (asked < r1) {
                const bool late = CUT && START && asked == 0 && l.t == 0, bottom = CUT && asked == a.rows - 1;
                const int upto = bottom ? l.C - 1 : l.C;
                R::ask(l, x, to + b * LINE, upto, late);
                if (block) R::ask(l, f, to + (RB + b) * LINE, upto, late);
                if (bottom && l.t == a.last_t && !(late && upto == 0)) {
                    const int at = a.last_v * a.tpr, slot = a.last_v * R::step;
                    R::ask_last(x + at, to + b * LINE + slot);
                    if (block) R::ask_last(f + at, to + (RB + b) * LINE + slot);
                }
                if (late) {
                    R::ask_first(x, to + b * LINE, upto == 0);
                    if (block) R::ask_first(f, to + (RB + b) * LINE, upto == 0);
                }
            }
            asked += a.slots;
            x += sx;
            f += sf;
        }
        copy_commit();
        to = to == ring + (D - 1) * STAGE ? ring : to + STAGE;
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) ask(std::true_type());
    float2 q[P], p[P], g2[P], b2[P];
    // pre's parameters: in registers, or, sixteen channels a thread, at a place of
    // the thread's own in shared memory (with 64 registers of parameters some
    // 130 bytes of a thread's were spilled: 4096x8192 bf16 63 us)
    float4 *const par = reinterpret_cast<float4 *>(smem + (size_t)D * 2 * RB * R::NV * blockDim.x * sizeof(Slot)) + threadIdx.x;
    auto pre = [&](float2 (&v)[P]) {
        if constexpr (K == 1) {
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = fma2(v[i], g2[i], b2[i]);
        } else {
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float4 g = par[i * blockDim.x], b = par[(i + 1) * blockDim.x];
                v[i] = fma2(v[i], make_float2(g.x, g.y), make_float2(b.x, b.y));
                v[i + 1] = fma2(v[i + 1], make_float2(g.z, g.w), make_float2(b.z, b.w));
            }
        }
    };
    int image = n;
    const bool by_row = RB == 1 && a.gate;
    if (by_row) image = min(row, a.rows - 1) / a.HW;
    if (block) factors(l, a, image, q, p);
    l.params(g2, a.g2, 1.0f);
    l.params(b2, a.b2, 0.0f);
    if constexpr (K > 1)
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            par[i * blockDim.x] = make_float4(g2[i].x, g2[i].y, g2[i + 1].x, g2[i + 1].y);
            par[(i + 1) * blockDim.x] = make_float4(b2[i].x, b2[i].y, b2[i + 1].x, b2[i + 1].y);
        }
    for (int base = r0; base < r1; base += a.slots * RB) {
        copy_wait<D - 2>();
        float2 v[RB][P], u[RB][P];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            R::get(l, d + b * LINE, ox + b * nx, v[b]);
            if (block) R::get(l, d + (RB + b) * LINE, of + b * nf, u[b]);
        }
        ox += RB * nx;
        of += RB * nf;
        d = d == ring + (D - 1) * STAGE ? ring : d + STAGE;
        ask(std::false_type());
        float2 one[RB], two[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) one[b] = two[b] = make_float2(0.0f, 1.0f);
        if (block) {
            if (by_row && row < r1) {
                const int k = row / a.HW;
                if (k != image) factors(l, a, image = k, q, p);
            }
            if (a.post != CONV_NORM_NONE) normalise<VEC, K, RB>(l, sum, u, a.post, a, one);
            if (ALL || a.b1)
#pragma unroll
                for (int b = 0; b < RB; ++b)
#pragma unroll
                    for (int i = 0; i < P; ++i) v[b][i] = add2(v[b][i], p[i]);
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int i = 0; i < P; ++i) v[b][i] = fma2(q[i], u[b][i], v[b][i]);
            if (ALL || a.o0)
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    if (row + b * a.slots < r1) R::put(l, y + b * sy, v[b]);
        }
        if (norm) {
            normalise<VEC, K, RB>(l, sum, v, a.pre, a, two);
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                pre(v[b]);
                if (row + b * a.slots < r1) R::put(l, z + b * sz, v[b]);
            }
        }
        if (a.stats && l.t == 0)
#pragma unroll
            for (int b = 0; b < RB; ++b)
                if (row + b * a.slots < r1) a.stats[row + b * a.slots] = make_float4(one[b].x, one[b].y, two[b].x, two[b].y);
        row += RB * a.slots;
        y += RB * sy;
        z += RB * sz;
    }
    copy_wait<0>();
}

// ------------------------------------------------------------------ host side
template <typename T, int VEC, bool CUT = false>
const void *pick_fwd(int k, int rb, int tpr, bool all) {
    if constexpr (sizeof(T) == 2 || VEC == 1)  // (fp32 rows of a warp and sixteen channels are ragged)
        if (k == 2 && tpr == 32) return all ? (const void *)&bn_fwd_kernel<T, VEC, 2, 1, ROW_WARP, true, CUT> : (const void *)&bn_fwd_kernel<T, VEC, 2, 1, ROW_WARP, false, CUT>;
    if (k == 2) return all ? (const void *)&bn_fwd_kernel<T, VEC, 2, 1, ROW_WARPS, true, CUT> : (const void *)&bn_fwd_kernel<T, VEC, 2, 1, ROW_WARPS, false, CUT>;
    if (rb == 1) return (const void *)&bn_fwd_kernel<T, VEC, 1, 1, ROW_ANY, false, CUT>;
    if (!all) return (const void *)&bn_fwd_kernel<T, VEC, 1, 2, ROW_ANY, false, CUT>;
    return tpr < 32 ? (const void *)&bn_fwd_kernel<T, VEC, 1, 2, ROW_PART, true, CUT>
                    : (tpr == 32 ? (const void *)&bn_fwd_kernel<T, VEC, 1, 2, ROW_WARP, true, CUT> : (const void *)&bn_fwd_kernel<T, VEC, 1, 2, ROW_WARPS, true, CUT>);
}
// (rb: rows at a time of the forward kernel, 0: the gradient)
const void *pick_kernel(conv_dtype_t dt, int vec, bool cut, const BnGeom::Part &d, bool all) {
    using B = __nv_bfloat16;
    const int rb = d.rb, k = d.k, tpr = d.tpr;
    if (!rb) return bn::pick_bwd(dt, vec, cut, d.pair, tpr, all);
    if (dt == CONV_F32) return vec == 4 ? pick_fwd<float, 4>(k, rb, tpr, all) : pick_fwd<float, 1>(k, rb, tpr, all);
    if (vec > 1) return vec == 8 ? pick_fwd<B, 8>(k, rb, tpr, all) : pick_fwd<B, 2>(k, rb, tpr, all);
    return cut ? pick_fwd<B, 1, true>(k, rb, tpr, all) : pick_fwd<B, 1>(k, rb, tpr, all);
}

// Channels a vector access takes: the widest that the channel count, every
// map's pitch and every map's address allow (a null map: any).
struct Map { const void *p; long long pitch; };
template <int N>
int vec_for(const conv_plan *p, const Map (&maps)[N]) {
    const int es = conv_esize(p->dtype);
    const int widths[2] = {16 / es, p->dtype == CONV_F32 ? 1 : 2};
    for (int v : widths) {
        bool ok = p->s.c_in % v == 0;
        for (const Map &m : maps) ok = ok && (!m.p || (m.pitch % v == 0 && (uintptr_t)m.p % (uintptr_t)(v * es) == 0));
        if (ok) return v;
    }
    return 1;
}

// Whether one of the maps of single bf16 values starts in the middle of a 4-byte word
// or ends in one.
template <int N>
bool cuts_words(const conv_plan *p, const Map (&maps)[N]) {
    const long long rows = (long long)p->s.n * p->s.h * p->s.w;
    for (const Map &m : maps)
        if (m.p && (((uintptr_t)m.p | ((uintptr_t)m.p + 2 * ((rows - 1) * m.pitch + p->s.c_in))) & 3u)) return true;
    return false;
}

long long up(long long a, long long b) { return (a + b - 1) / b; }

// Bytes of the ring of a CTA: a thread's 8 k channels of each map and stage.
// (The gradient's holds the sums of rows side by side after its last row: it has
// 96 elements a thread where the sums are SUMS * 8 in fp32.
// A cluster's also holds the CTA's sums of its channels, at most 8 a thread of a
// row, and there are rows side by side where that is at most half of them: 64.)
static_assert(3 * 4 * 8 * 2 >= SUMS * 8 * 4 + SUMS * 8 * 4 / 2, "");
// es: of an element in the ring.
size_t ring_bytes(const BnGeom::Part &d, int es) {
    const size_t maps = (size_t)d.threads * 8 * d.k * es;
    if (d.rb) return 2 * fwd_stages(es, d.k) * d.rb * maps + (d.k > 1 ? (size_t)d.threads * 2 * 8 * d.k * 4 : 0);
    return bwd_stages() * (4 * maps + (size_t)d.threads / (d.tpr < 32 ? d.tpr : 32) * 16);  // (and a row's statistics)
}

// in: the maps that are read.
template <int N>
cudaError_t launch(const conv_plan *p, const BnGeom::Part &d, int vec, const Map (&in)[N], BnArgs &a, cudaStream_t st) {
    const size_t smem = ring_bytes(d, ring_element(conv_esize(p->dtype), vec));
    const void *k = pick_kernel(p->dtype, vec, cuts_words(p, in), d, d.rb ? a.f && a.o0 && a.o1 : a.f && a.dy && a.dz);
    if (smem > 40 * 1024) {  // (with the kernel's static shared memory: 48 KB are free)
        const int rc = conv_grant_smem_once(k, p->device, (int)smem);
        if (rc != CONV_OK) return cudaErrorInvalidValue;
    }
    if (d.joined && conv_allow_cluster_once(k, p->device, d.grid) != CONV_OK) return cudaErrorInvalidValue;
    const int last = (a.C - 1) / d.tpr, vectors = 8 * d.k;
    a.last_v = last % vectors; a.last_t = (a.C - 1) % d.tpr + (last - a.last_v) * d.tpr;
    a.tpr = d.tpr; a.full = d.full; a.slots = d.slots; a.run = d.run; a.S = d.S; a.units = d.units; a.whole = d.whole; a.joined = d.joined;
    void *args[] = {&a};
    return conv_launch(k, dim3((unsigned)d.grid << d.pair), dim3((unsigned)d.threads), args, smem, st, d.joined ? d.grid : 1 << d.pair);
}

int check_map(const conv_plan *p, const void *t, int64_t *pitch) {
    if (!t) return CONV_OK;
    if (*pitch == 0) *pitch = p->s.c_in;
    if (*pitch < p->s.c_in) return CONV_ERR_INVALID_ARG;
    if (*pitch >= (1ll << 31) || (long long)p->s.n * p->s.h * p->s.w * *pitch >= (1ll << 40)) return CONV_ERR_UNSUPPORTED;
    if ((uintptr_t)t % (uintptr_t)conv_esize(p->dtype)) return CONV_ERR_MISALIGNED;
    return CONV_OK;
}

// Whether a buffer that a run writes shares a byte with another that it reads
// or writes.  A written map may be an input map itself (every element is read
// by the thread that writes it, before it does), not otherwise overlap it.
struct Small { const void *p; size_t bytes; };
template <int M, int W, int I, int O>
bool shared(const Map (&in)[M], const Map (&out)[W], const Small (&small_in)[I], const Small (&small_out)[O], long long rows,
            int C, int es) {
    for (int i = 0; i < W; ++i) {
        for (const Map &m : in)
            if (!(m.p == out[i].p && m.pitch == out[i].pitch) && maps_overlap(m.p, m.pitch, out[i].p, out[i].pitch, rows, C, es))
                return true;
        for (int j = 0; j < i; ++j)
            if (maps_overlap(out[j].p, out[j].pitch, out[i].p, out[i].pitch, rows, C, es)) return true;
        for (const Small &s : small_in)
            if (range_overlaps(s.p, s.bytes, out[i].p, out[i].pitch, rows, C, es)) return true;
    }
    for (int i = 0; i < O; ++i) {
        const Small &s = small_out[i];
        for (const Map &m : in)
            if (range_overlaps(s.p, s.bytes, m.p, m.pitch, rows, C, es)) return true;
        for (const Map &m : out)
            if (range_overlaps(s.p, s.bytes, m.p, m.pitch, rows, C, es)) return true;
        for (const Small &t : small_in)
            if (conv_overlaps(s.p, s.bytes, t.p, t.bytes)) return true;
        for (int j = 0; j < i; ++j)
            if (conv_overlaps(s.p, s.bytes, small_out[j].p, small_out[j].bytes)) return true;
    }
    return false;
}
bool bad_f32(const void *t) { return t && ((uintptr_t)t & 3u); }

// All rows in runs of whole sets of rows side by side, one wave of CTAs.
void divide_rows(BnGeom::Part &d, long long rows, long long set, long long wave) {
    long long run = up(up(rows, wave), set) * set;
    if (run < set) run = set;
    d.run = (int)run;
    d.S = d.units = d.grid = (int)up(rows, run);
    d.whole = d.joined = 0;
}
// Each image in runs of whole sets, as many as fill the CTAs best: a run costs
// its sets and about four more for its start and end.
void divide_images(BnGeom::Part &d, long long N, long long HW, long long set, long long wave) {
    long long best = -1;
    for (long long S = 1; S <= 1024; ++S) {
        const long long sets = up(up(HW, S), set);
        if (S > 1 && up(HW, sets * set) != S) continue;
        const long long cost = up(N * S, wave) * (sets + 4);
        if (best >= 0 && cost >= best) continue;
        best = cost;
        d.S = (int)S;
        d.run = (int)(S == 1 ? HW : sets * set);
    }
    d.units = d.grid = (int)(N * d.S);
    d.whole = d.joined = 0;
}

// Threads of a row, rows of a CTA, and how the rows are divided.
void plan_geometry(conv_plan *p) {
    BnGeom &g = p->bn;
    const int C = p->s.c_in, es = conv_esize(p->dtype);
    const long long N = p->s.n, HW = (long long)p->s.h * p->s.w, rows = N * HW;
    p->ws_bytes = p->ws_bwd_bytes = 0;
    if (rows == 0) return;
    auto part = [&](BnGeom::Part &d, int rb, int k, int threads, int pair = 0) {
        d.rb = rb;
        d.k = k;
        d.pair = pair;
        const int one = 8 * k << pair, want = (C + one - 1) / one;
        d.tpr = 1;
        if (want > 32) d.tpr = (want + 31) / 32 * 32;
        else while (d.tpr < want) d.tpr *= 2;
        d.full = C == d.tpr * one;
        d.slots = d.tpr <= threads ? threads / d.tpr : 1;
        d.threads = d.tpr * d.slots;
    };
    // CTAs of one wave: 512 threads a SM, where their rings fit
    auto wave = [&](const BnGeom::Part &d) {
        const long long smem = (228 * 1024) / (long long)(ring_bytes(d, es) + 1024 + 256), regs = kMostThreads / d.threads;
        const long long n = smem < regs ? smem : regs;
        return ((long long)p->num_sms * (n < 1 ? 1 : n)) >> d.pair;
    };
    // sixteen channels a thread, forward: beyond 2048, where eight leave one CTA a
    // SM, and beyond 4096 would take more threads than a CTA has registers for
    // (6144x2560 bf16 36 us, with sixteen 27; 8192x4096 55 and 51; below, 4096x2048
    // 16.5 and 15.7, 3200x1024 7.2 and 7.7).  The gradient keeps to eight (58 and 84,
    // 91 and 133) and gives a row beyond 4096 to two CTAs of a cluster (4096x8192 bf16
    // 98 us, 2048x8192 fp32 73, where sixteen took 147 and 117; up to 4096 a CTA
    // holds it: 8192x4096 bf16 84, a pair 97, 4096x4096 fp32 71 and 71, 8192x2560
    // bf16 70 and 67).
    // From 257 to 512 channels sixteen make a row a warp's, whose sums need no barrier.
    // That pays for more rows than four sets of eight channels a thread (4864 on 152
    // SMs), of maps whose channels are no whole 16-byte vectors, and of bf16 without a
    // gate under a layer norm.  Eight and sixteen, us, ungated:
    //   rows                     2432          4864          12800         51200
    //   510 bf16 layer, rms      4.2, 4.8      6.3, 6.5      16.4, 15.3    48.5, 44.8
    //   511 bf16 rms, rms        5.2, 5.9      8.4, 8.4      21.7, 20.2    67.5, 61.1
    //   511 fp32 layer, layer    5.5, 6.3      12.0, 12.1    26.8, 24.8    86.5, 80.0
    //   264 bf16 layer, rms      3.5, 4.0      5.2, 5.4      11.9, 10.8    38.0, 32.5
    //   512 bf16 layer, layer    4.0, 4.7      6.0, 6.4      14.6, 14.1    42.8, 37.9
    //   512 bf16 layer, rms      3.7, 4.4      5.4, 5.9      13.2, 13.2    38.0, 39.5
    //   512 bf16 rms, rms        3.3, 4.1      4.8, 5.5      11.7, 12.4    36.4, 39.7
    // and with a gate at 12800 rows: 511 bf16 layer, rms 23.2, 22.9; 512 13.3, 14.8.
    // (Slices at addresses that allow no vectors go by their channel count all the
    // same: 512 of 513 bf16 rms, rms at 12800 rows 21.8, 19.5.)
    const bool layers = g.post == CONV_NORM_LAYER || g.pre == CONV_NORM_LAYER, ragged = C * es % 16 != 0;
    part(g.fwd, 1, 1, kThreads);
    const bool many = C > 256 && C <= 512 && rows > 4 * wave(g.fwd) * g.fwd.slots;
    const int pair = C > 8 * kMostThreads;
    // two rows at a time where one wave of CTAs takes more than one set of rows
    // (64x25x5x61 fp32, 0.8 of a set: one at a time 4.5 us, two 5.7)
    auto forward = [&](BnGeom::Part &d, bool sixteen) {
        part(d, 1, sixteen ? 2 : 1, kThreads);
        if (!sixteen && rows > wave(d) * d.slots) d.rb = 2;
    };
    forward(g.fwd, C > 2048 || (many && (ragged || (es == 2 && layers))));
    forward(g.fwd_gated, C > 2048 || (many && ragged));
    divide_rows(g.fwd, rows, (long long)g.fwd.slots * g.fwd.rb, wave(g.fwd));
    if (g.fwd_gated.rb == 2 && HW >= 4LL * g.fwd_gated.slots) divide_images(g.fwd_gated, N, HW, 2LL * g.fwd_gated.slots, wave(g.fwd_gated));
    else {
        g.fwd_gated.rb = 1;
        divide_rows(g.fwd_gated, rows, g.fwd_gated.slots, wave(g.fwd_gated));
    }
    // the gradient in large CTAs: a part of the sums from each
    part(g.bwd, 0, 1, pair ? 1 : kMostThreads, pair);
    g.bwd_gated = g.bwd;
    // (images of fewer rows than lie side by side: smaller CTAs, more of them.
    // 2048 images of one pixel of 1024 channels, bf16: 90 us in CTAs of 512, 50 so)
    if (HW < g.bwd.slots) part(g.bwd_gated, 0, 1, (int)up(g.bwd.tpr * HW, 32) * 32);
    const long long w = wave(g.bwd_gated);
    divide_rows(g.bwd, rows, g.bwd.slots, wave(g.bwd));
    divide_images(g.bwd_gated, N, HW, g.bwd_gated.slots, w);
    // few rows: the CTAs of one cluster, a unit each, which join their sums
    // themselves, where none takes more than two sets of rows (2x7x7x512: the call
    // 14 us on the host and 8.5 on the device; in two launches 19 and 7.1)
    auto cluster = [&](BnGeom::Part &d, long long images, long long each) {
        const long long most = images <= kCluster ? kCluster / images : 0, sets = most ? up(each, most * d.slots) : 0;
        if (pair || !most || sets > kClusterSets) return;
        const long long run = sets * d.slots, S = up(each, run);
        // (of the instances that a call may choose, the one of the widest vectors
        // stands for all, with the shared memory of the one that takes the most)
        const void *kernel = pick_kernel(p->dtype, 16 / es, false, d, true);
        const size_t smem = ring_bytes(d, 4);
        if (conv_grant_smem_once(kernel, p->device, (int)smem) != CONV_OK ||
            !conv_cluster_fits(kernel, p->device, (int)(images * S), d.threads, smem))
            return;
        d.run = (int)run;
        d.S = (int)S;
        d.units = d.grid = (int)(images * S);
        d.joined = 1;
    };
    cluster(g.bwd, 1, rows);
    cluster(g.bwd_gated, N, HW);
    if (!g.bwd_gated.joined) {
        g.bwd_gated.whole = g.bwd_gated.S == 1;
        if (g.bwd_gated.whole && N > w) g.bwd_gated.grid = (int)w;
    }
    const long long open = g.bwd.joined ? 0 : g.bwd.grid, gated = g.bwd_gated.joined ? 0 : g.bwd_gated.grid;
    const long long parts = open > gated ? open : gated;
    p->ws_bwd_bytes = (size_t)parts * SUMS * ((C + 3) / 4 * 4) * 4;
}

}  // namespace

extern "C" int conv_plan_create_blocknorm(int32_t n, int32_t h, int32_t w, int32_t c, conv_norm_t post, conv_norm_t pre,
                                          float eps, conv_dtype_t dtype, conv_plan_t **out_plan) {
    if (!out_plan) return CONV_ERR_NULL_ARG;
    *out_plan = nullptr;
    if (n < 0 || h < 1 || w < 1 || c < 1) return CONV_ERR_INVALID_SHAPE;
    if ((int)dtype < CONV_F32 || (int)dtype > CONV_I8) return CONV_ERR_INVALID_ARG;
    if ((int)post < CONV_NORM_NONE || (int)post > CONV_NORM_RMS || (int)pre < CONV_NORM_NONE || (int)pre > CONV_NORM_RMS)
        return CONV_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !isfinite(eps)) return CONV_ERR_INVALID_ARG;
    if (dtype == CONV_I8) return CONV_ERR_UNSUPPORTED;
    // 32-bit pixel indices, a row's channels in one CTA
    if (c > kMaxC || (long long)h * w >= (1ll << 30) || (long long)h * w * n >= (1ll << 30)) return CONV_ERR_UNSUPPORTED;
    conv_plan *p = new (std::nothrow) conv_plan();
    if (!p) return CONV_ERR_OOM;
    p->s = {n, h, w, c, c, 1, 1};
    p->stride = 1; p->groups = 1; p->dtype = dtype; p->oh = h; p->ow = w;
    p->y_c = c; p->up = 1; p->algo = CONV_ALGO_BLOCKNORM;
    p->bn.post = post; p->bn.pre = pre; p->bn.eps = eps;
    const int rc = conv_plan_bind_device(p, false);
    if (rc != CONV_OK) {
        conv_plan_destroy(p);
        return rc;
    }
    plan_geometry(p);
    static const char *const names[] = {"none", "layer", "rms"};
    snprintf(p->desc, sizeof(p->desc), "blocknorm %s post=%s pre=%s threads=%dx%d channels/thread=%d ctas=%d gradient: %d, gated %d in %d",
             dtype == CONV_F32 ? "f32" : "bf16", names[post], names[pre], p->bn.fwd.slots, p->bn.fwd.tpr, 8 * p->bn.fwd.k, p->bn.fwd.grid,
             p->bn.bwd.grid, p->bn.bwd_gated.units, p->bn.bwd_gated.grid);
    *out_plan = p;
    return CONV_OK;
}

namespace {
BnArgs base_args(const conv_plan *p, const conv_blocknorm_params_t &w, const void *x, int64_t px, const void *f, int64_t pf) {
    BnArgs a = {};
    a.x = x; a.px = px; a.f = f; a.pf = pf;
    a.scale = w.scale; a.gate = w.gate; a.g1 = w.post_gamma; a.b1 = w.post_beta; a.g2 = w.pre_gamma; a.b2 = w.pre_beta;
    a.eps = p->bn.eps; a.inv_c = 1.0f / (float)p->s.c_in;
    a.N = p->s.n; a.HW = p->s.h * p->s.w; a.rows = a.N * a.HW; a.C = p->s.c_in; a.Cp = (a.C + 3) / 4 * 4;
    a.post = p->bn.post; a.pre = p->bn.pre;
    return a;
}
int check_params(const conv_plan *p, const conv_blocknorm_params_t &w, const void *f) {
    if (!f && (w.scale || w.gate || w.post_gamma || w.post_beta || p->bn.post != CONV_NORM_NONE)) return CONV_ERR_INVALID_ARG;
    if (p->bn.post == CONV_NORM_NONE && (w.post_gamma || w.post_beta)) return CONV_ERR_INVALID_ARG;
    if (p->bn.pre == CONV_NORM_NONE && (w.pre_gamma || w.pre_beta)) return CONV_ERR_INVALID_ARG;
    if (bad_f32(w.scale) || bad_f32(w.gate) || bad_f32(w.post_gamma) || bad_f32(w.post_beta) || bad_f32(w.pre_gamma) ||
        bad_f32(w.pre_beta))
        return CONV_ERR_MISALIGNED;
    return CONV_OK;
}
}  // namespace

extern "C" int conv_run_blocknorm(const conv_plan_t *plan, const void *x, int64_t x_pitch, const void *f, int64_t f_pitch,
                                  const conv_blocknorm_params_t *params, void *y, int64_t y_pitch, void *z, int64_t z_pitch,
                                  float *stats, void *stream) {
    if (!plan) return CONV_ERR_NULL_ARG;
    const conv_plan *p = plan;
    if (p->algo != CONV_ALGO_BLOCKNORM) return CONV_ERR_INVALID_ARG;
    if (p->s.n == 0) return CONV_OK;
    static const conv_blocknorm_params_t kNone = {};
    const conv_blocknorm_params_t &w = params ? *params : kNone;
    const bool norm = p->bn.pre != CONV_NORM_NONE;
    if (!x || (norm && !z) || (!norm && !y)) return CONV_ERR_NULL_ARG;
    if ((!norm && z) || (!f && y)) return CONV_ERR_INVALID_ARG;
    int rc;
    if ((rc = check_params(p, w, f)) != CONV_OK || (rc = check_map(p, x, &x_pitch)) != CONV_OK ||
        (rc = check_map(p, f, &f_pitch)) != CONV_OK || (rc = check_map(p, y, &y_pitch)) != CONV_OK ||
        (rc = check_map(p, z, &z_pitch)) != CONV_OK)
        return rc;
    if ((uintptr_t)stats & 15u) return CONV_ERR_MISALIGNED;
    const int es = conv_esize(p->dtype), C = p->s.c_in;
    const long long rows = (long long)p->s.n * p->s.h * p->s.w;
    const size_t cb = (size_t)C * 4, nb = (size_t)p->s.n * cb;
    const Map in[2] = {{x, x_pitch}, {f, f_pitch}}, out[2] = {{y, y_pitch}, {z, z_pitch}};
    const Small si[6] = {{w.scale, cb}, {w.gate, nb}, {w.post_gamma, cb}, {w.post_beta, cb}, {w.pre_gamma, cb}, {w.pre_beta, cb}};
    const Small so[1] = {{stats, (size_t)rows * 16}};
    if (shared(in, out, si, so, rows, C, es)) return CONV_ERR_ALIASING;
    BnArgs a = base_args(p, w, x, x_pitch, f, f_pitch);
    a.o0 = y; a.p0 = y_pitch; a.o1 = z; a.p1 = z_pitch;
    a.stats = reinterpret_cast<float4 *>(stats);
    const Map all[4] = {in[0], in[1], out[0], out[1]};
    const BnGeom::Part &g = w.gate ? p->bn.fwd_gated : p->bn.fwd;
    return launch(p, g, vec_for(p, all), in, a, (cudaStream_t)stream) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

extern "C" int conv_run_blocknorm_bwd(const conv_plan_t *plan, const void *x, int64_t x_pitch, const void *f, int64_t f_pitch,
                                      const conv_blocknorm_params_t *params, const float *stats, const void *dy,
                                      int64_t dy_pitch, const void *dz, int64_t dz_pitch, void *dx, int64_t dx_pitch,
                                      void *df, int64_t df_pitch, const conv_blocknorm_grads_t *grads, void *workspace,
                                      void *stream) {
    if (!plan) return CONV_ERR_NULL_ARG;
    const conv_plan *p = plan;
    if (p->algo != CONV_ALGO_BLOCKNORM) return CONV_ERR_INVALID_ARG;
    static const conv_blocknorm_params_t kNone = {};
    static const conv_blocknorm_grads_t kNoGrads = {};
    const conv_blocknorm_params_t &w = params ? *params : kNone;
    const conv_blocknorm_grads_t &d = grads ? *grads : kNoGrads;
    cudaStream_t st = (cudaStream_t)stream;
    const int es = conv_esize(p->dtype), C = p->s.c_in;
    const size_t cb = (size_t)C * 4;
    if (bad_f32(d.scale) || bad_f32(d.gate) || bad_f32(d.post_gamma) || bad_f32(d.post_beta) || bad_f32(d.pre_gamma) ||
        bad_f32(d.pre_beta))
        return CONV_ERR_MISALIGNED;
    if ((p->bn.post == CONV_NORM_NONE && (d.post_gamma || d.post_beta)) || (p->bn.pre == CONV_NORM_NONE && (d.pre_gamma || d.pre_beta)))
        return CONV_ERR_INVALID_ARG;
    if (p->s.n == 0) {  // sums over nothing (a gate has no rows)
        float *const sums[5] = {d.scale, d.post_gamma, d.post_beta, d.pre_gamma, d.pre_beta};
        for (float *s : sums)
            if (s && cudaMemsetAsync(s, 0, cb, st) != cudaSuccess) return CONV_ERR_CUDA;
        return CONV_OK;
    }
    const bool norm = p->bn.pre != CONV_NORM_NONE;
    if (!x || !dx || (norm && !dz) || (!norm && !dy) || !stats || (f && !df)) return CONV_ERR_NULL_ARG;
    if ((!norm && dz) || (!f && (df || d.scale || d.gate)) || (d.gate && !w.gate)) return CONV_ERR_INVALID_ARG;
    int rc;
    if ((rc = check_params(p, w, f)) != CONV_OK || (rc = check_map(p, x, &x_pitch)) != CONV_OK ||
        (rc = check_map(p, f, &f_pitch)) != CONV_OK || (rc = check_map(p, dy, &dy_pitch)) != CONV_OK ||
        (rc = check_map(p, dz, &dz_pitch)) != CONV_OK || (rc = check_map(p, dx, &dx_pitch)) != CONV_OK ||
        (rc = check_map(p, df, &df_pitch)) != CONV_OK)
        return rc;
    if (((uintptr_t)stats & 15u) || ((uintptr_t)workspace & 15u)) return CONV_ERR_MISALIGNED;
    if (p->ws_bwd_bytes && !workspace) return CONV_ERR_NULL_ARG;
    const long long rows = (long long)p->s.n * p->s.h * p->s.w;
    const size_t nb = (size_t)p->s.n * cb;
    const Map in[4] = {{x, x_pitch}, {f, f_pitch}, {dy, dy_pitch}, {dz, dz_pitch}}, out[2] = {{dx, dx_pitch}, {df, df_pitch}};
    const Small si[7] = {{w.scale, cb}, {w.gate, nb}, {w.post_gamma, cb}, {w.post_beta, cb}, {w.pre_gamma, cb}, {w.pre_beta, cb},
                         {stats, (size_t)rows * 16}};
    const Small so[7] = {{d.scale, cb}, {d.gate, nb}, {d.post_gamma, cb}, {d.post_beta, cb}, {d.pre_gamma, cb}, {d.pre_beta, cb},
                         {workspace, p->ws_bwd_bytes}};
    if (shared(in, out, si, so, rows, C, es)) return CONV_ERR_ALIASING;
    BnArgs a = base_args(p, w, x, x_pitch, f, f_pitch);
    a.dy = dy; a.pdy = dy_pitch; a.dz = dz; a.pdz = dz_pitch;
    a.o0 = dx; a.p0 = dx_pitch; a.o1 = df; a.p1 = df_pitch;
    a.stats = reinterpret_cast<float4 *>(const_cast<float *>(stats));
    a.part = static_cast<float *>(workspace);
    a.dscale = d.scale; a.dgate = d.gate; a.dg1 = d.post_gamma; a.db1 = d.post_beta; a.dg2 = d.pre_gamma; a.db2 = d.pre_beta;
    a.want_b = d.post_beta || (w.post_beta && (d.scale || d.gate));
    const BnGeom::Part &g = w.gate ? p->bn.bwd_gated : p->bn.bwd;
    const Map all[6] = {in[0], in[1], in[2], in[3], out[0], out[1]};
    if (launch(p, g, vec_for(p, all), in, a, st) != cudaSuccess) return CONV_ERR_CUDA;
    const bool sums = d.scale || d.post_gamma || d.post_beta || d.pre_gamma || d.pre_beta, images = d.gate && !g.whole;
    if (g.joined || (!sums && !images)) return CONV_OK;
    return launch_join(a, g.grid, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}
