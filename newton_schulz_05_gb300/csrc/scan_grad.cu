// Gradient of the gated linear recurrence: the same joins from the last token to the
// first, over what reaches the state behind each token, c -> a (dh + c).
#include "scan.cuh"

namespace muon {

namespace {

struct ScanBwd {
  int64_t length, dim, lddh, ldg, ldx, ldh;
  int strips;
  float mix;          // 1 or 0: how much of x the state's difference has
  const void *dh, *gate, *x, *h;
  const float *state, *dlast;
  const uint8_t *starts, *mask;
  void *dgate, *dx;
  float* dstate;
};

template <typename T, int W, int S, int CL, int D, bool VEC, bool FLAGS>
__global__ void __launch_bounds__(32 * W, W >= 8 ? 2 : 16 / W)
scan_bwd_kernel(const __grid_constant__ ScanBwd a) {
  extern __shared__ uint4 ring[];
  __shared__ RunSlots<W, CL> sh;
  pdl_wait();
  constexpr int kSpan = 2 * W * S, NT = 32 * W;
  const int rank = CL > 1 ? cluster_rank() : 0;      // rank 0 has the last chunk
  const int64_t unit = blockIdx.x / CL, b = unit / a.strips;
  const Channels<VEC> ch((int)(unit % a.strips), a.dim);
  const int64_t row0 = b * a.length;
  const T* dh = static_cast<const T*>(a.dh) + row0 * a.lddh + ch.first;
  const T* gate = static_cast<const T*>(a.gate) + row0 * a.ldg + ch.first;
  const T* x = static_cast<const T*>(a.x) + row0 * a.ldx + ch.first;
  const T* h = static_cast<const T*>(a.h) + row0 * a.ldh + ch.first;
  T* dg = static_cast<T*>(a.dgate) + row0 * a.dim + ch.first;
  T* dx = static_cast<T*>(a.dx) + row0 * a.dim + ch.first;
  const bool mix = a.mix != 0.f;
  Quad carry = a.dlast ? ch.state(a.dlast + b * a.dim + ch.first) : quad(0.f);
  const int seg = threadIdx.x >> 4;
  Raw4<T>* const slots = reinterpret_cast<Raw4<T>*>(ring) + threadIdx.x;
  Flags ahead[D > 0 ? D : 1];
  const int64_t chunks = (a.length + kSpan - 1) / kSpan, stride = (int64_t)kSpan * CL;
  const int64_t first = (chunks - 1 - rank) * kSpan + seg * S;
  auto start = [&](int64_t t0, int stage) {
    #pragma unroll
    for (int i = 0; i < S; ++i) {
      const int64_t t = t0 + i;
      Raw4<T>* const to = slots + (stage * 4 * S + i) * NT;
      if (t >= 0 && t < a.length && ch.any()) {
        ch.copy(to, dh + t * a.lddh);
        ch.copy(to + S * NT, gate + t * a.ldg);
        if (mix) ch.copy(to + 2 * S * NT, x + t * a.ldx);
        else zero(to[2 * S * NT]);
        if (t > 0) ch.copy(to + 3 * S * NT, h + (t - 1) * a.ldh);
        else zero(to[3 * S * NT]);
      } else {
        zero(to[0]);
        infinite(to[S * NT]);
        zero(to[2 * S * NT]);
        zero(to[3 * S * NT]);
      }
    }
    copies_commit();
  };
  #pragma unroll
  for (int d = 0; d < D; ++d) {
    start(first - d * stride, d);
    if (FLAGS) ahead[d] = ask<S>(a.starts, a.mask, row0, first - d * stride, a.length);
  }
  if (CL > 1) cluster_barrier();      // every block has begun before one writes to another
  int round = 0, stage = 0;
  int64_t t0 = first;
  for (int64_t done = 0; done < chunks; done += CL, t0 -= stride, ++round) {
    if (FLAGS && D == 0) ahead[0] = ask<S>(a.starts, a.mask, row0, t0, a.length);
    Raw4<T> rd[S], rg[S], rx[S], rh[S];
    if constexpr (D > 0) {
      copies_wait<D - 1>();
    } else {
      #pragma unroll
      for (int i = 0; i < S; ++i) {
        const int64_t t = t0 + i;
        zero(rd[i]);
        infinite(rg[i]);
        zero(rx[i]);
        zero(rh[i]);
        if (t >= 0 && t < a.length && ch.any()) {
          ch.load(rd[i], dh + t * a.lddh);
          ch.load(rg[i], gate + t * a.ldg);
          if (mix) ch.load(rx[i], x + t * a.ldx);
          if (t > 0) ch.load(rh[i], h + (t - 1) * a.ldh);
        }
      }
    }
    Quad keep[S], take[S], d[S], v[S];
    Run run = {quad(1.f), quad(0.f), false};       // m: the factor, until the end
    Quad lost = quad(0.f);                          // 1 minus it
    const Flags now = FLAGS ? bits(ahead[0]) : Flags{0, 0};
    #pragma unroll
    for (int i = S - 1; i >= 0; --i) {
      Raw4<T> di, gi, xi, hi;
      if constexpr (D > 0) {
        const Raw4<T>* const from = slots + (stage * 4 * S + i) * NT;
        di = from[0];
        gi = from[S * NT];
        xi = from[2 * S * NT];
        hi = from[3 * S * NT];
      } else {
        di = rd[i];
        gi = rg[i];
        xi = rx[i];
        hi = rh[i];
      }
      if (FLAGS && !(now.live >> i & 1)) infinite(gi);
      const Quad g = widen(gi);
      #pragma unroll
      for (int j = 0; j < 2; ++j) {
        // t = 4 exp(-gate); a = 1 / (1 + t / 4), 1 - a = a t / 4, so that both have their
        // own precision.  The 4 makes t infinite before a is flushed to 0, and the minimum
        // drops the NaN of infinity times 0.
        float2 t = fma2(g.v[j], both(-1.4426950408889634f), both(2.f));
        t = make_float2(exp2_fast(t.x), exp2_fast(t.y));
        const float2 n = fma2(t, both(0.25f), both(1.f));
        keep[i].v[j] = make_float2(reciprocal_fast(n.x), reciprocal_fast(n.y));
        t = mul2(mul2(t, both(0.25f)), keep[i].v[j]);
        take[i].v[j] = make_float2(fminf(t.x, 1.f), fminf(t.y, 1.f));
      }
      d[i] = widen(di);
      v[i] = widen(hi);
      if (t0 + i == 0 && a.state && ch.any()) v[i] = ch.state(a.state + b * a.dim + ch.first);
      if (FLAGS && (now.starts >> i & 1)) v[i] = quad(0.f);
      v[i] = fma(widen(xi), quad(-a.mix), v[i]);
      run.m = mul(run.m, keep[i]);
      run.H = mul(keep[i], add(run.H, d[i]));
      lost = fma(keep[i], lost, take[i]);
      if (FLAGS && (now.starts >> i & 1)) {
        run.m = run.H = quad(0.f);
        run.cut = true;
      }
    }
    run.m = shares(run.m, lost);
    if constexpr (D > 0) {
      start(t0 - D * stride, stage);
      stage = stage + 1 == D ? 0 : stage + 1;
      if (FLAGS) {
        #pragma unroll
        for (int k = 0; k + 1 < D; ++k) ahead[k] = ahead[k + 1];
        ahead[D - 1] = ask<S>(a.starts, a.mask, row0, t0 - D * stride, a.length);
      }
    }
    Quad c = join_runs<W, CL, FLAGS, true>(sh, run, carry, round);
    #pragma unroll
    for (int i = S - 1; i >= 0; --i) {
      const Quad l = add(d[i], c), u = mul(take[i], l);
      c = mul(keep[i], l);
      Quad gx = mix ? u : l, gg = mul(mul(u, keep[i]), v[i]);
      if (FLAGS && !(now.live >> i & 1)) gx = gg = quad(0.f);
      if (t0 + i >= 0 && t0 + i < a.length && ch.any()) {
        if (a.dx) ch.store(dx + (t0 + i) * a.dim, gx);
        if (a.dgate) ch.store(dg + (t0 + i) * a.dim, gg);
      }
      if (FLAGS && (now.starts >> i & 1)) c = quad(0.f);
    }
  }
  if (a.dstate && rank == 0 && seg == 0) ch.put_state(a.dstate + b * a.dim + ch.first, carry);
}

template <typename T, int W, int S, int CL, int D, bool VEC>
cudaError_t scan_bwd_with(const ScanBwd& a, int64_t strips, cudaStream_t s) {
  constexpr size_t smem = (size_t)D * 4 * S * 32 * W * sizeof(Raw4<T>);
  constexpr auto plain = scan_bwd_kernel<T, W, S, CL, D, VEC, false>,
                 flags = scan_bwd_kernel<T, W, S, CL, D, VEC, true>;
  if (a.starts || a.mask) {
    if (const cudaError_t e = smem ? allow_shared<flags>(smem) : cudaSuccess) return e;
    return launch_strips<CL>(flags, strips, 32 * W, smem, s, a);
  }
  if (const cudaError_t e = smem ? allow_shared<plain>(smem) : cudaSuccess) return e;
  return launch_strips<CL>(plain, strips, 32 * W, smem, s, a);
}

template <typename T, bool VEC> cudaError_t scan_bwd_by_size(const ScanBwd& a, int64_t strips, cudaStream_t s) {
  constexpr int S = sizeof(T) == 2 ? 4 : 2, D = VEC ? 3 : 0;
  if (a.length <= 2 * S) return scan_bwd_with<T, 1, S, 1, 0, VEC>(a, strips, s);
  if (a.length <= 8 * S) return scan_bwd_with<T, 4, S, 1, 0, VEC>(a, strips, s);
  if (strips >= 304 || a.length <= 16 * S) return scan_bwd_with<T, 8, S, 1, D, VEC>(a, strips, s);
  if (strips >= 76 || a.length <= 64 * S) return scan_bwd_with<T, 8, S, 4, D, VEC>(a, strips, s);
  return scan_bwd_with<T, 8, S, 8, D, VEC>(a, strips, s);
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_gated_scan_backward(
    int64_t batch, int64_t length, int64_t dim, int dtype, const void* dh, int64_t lddh,
    const void* gate, int64_t ldg, const void* x, int64_t ldx, const void* h, int64_t ldh,
    const float* state, const float* dlast, const uint8_t* starts, const uint8_t* token_mask,
    int mix, void* dgate, void* dx, float* dstate, void* stream) {
  const muon_status st = check_scan(batch, length, dim, dtype);
  if (st != MUON_OK) return st;
  if (lddh < 0 || ldg < 0 || ldx < 0 || ldh < 0 ||
      (batch > 0 && length > 0 && (!dh || !gate || (mix && !x) || !h)))
    return MUON_ERR_INVALID_ARG;
  const size_t es = size_of(dtype);
  if (any_off(es, dh, gate, x, h, dgate, dx) || any_off(4, state, dlast, dstate))
    return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (batch == 0) return MUON_OK;
  NvtxRange range("muon_gated_scan_backward");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int strips = (int)((dim + kStrip - 1) / kStrip);
  const ScanBwd a = {length, dim, lddh, ldg, ldx, ldh, strips, mix ? 1.f : 0.f, dh, gate, x, h, state, dlast, starts,
                     token_mask, dgate, dx, dstate};
  const int64_t rows = batch * length;
  const bool vec = dim % 4 == 0 && fours(dh, rows, lddh, es) && fours(gate, rows, ldg, es) &&
                   (!mix || fours(x, rows, ldx, es)) && fours(h, rows, ldh, es) && !off(dgate, 4 * es) &&
                   !off(dx, 4 * es);
  const cudaError_t e = by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return vec ? scan_bwd_by_size<T, true>(a, batch * strips, s)
               : scan_bwd_by_size<T, false>(a, batch * strips, s);
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
