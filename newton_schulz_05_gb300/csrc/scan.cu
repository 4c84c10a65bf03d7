// Gated linear recurrence: the forward pass.
#include "scan.cuh"

namespace muon {

namespace {

struct Scan {
  int64_t length, dim, ldg, ldx;
  int strips;
  float mix;          // 1: the input is multiplied by 1 - a; 0: it is not
  const void *gate, *x;
  const float* state;
  const uint8_t *starts, *mask;
  void* h;
  float* last;
};

// W warps a block, S tokens a segment, CL blocks a cluster, D chunks in flight (0: a
// chunk is read when it is needed)
template <typename T, int W, int S, int CL, int D, bool VEC, bool FLAGS>
__global__ void __launch_bounds__(32 * W, W >= 8 ? 2 : 16 / W)
scan_kernel(const __grid_constant__ Scan a) {
  extern __shared__ uint4 ring[];
  __shared__ RunSlots<W, CL> sh;
  pdl_wait();
  constexpr int kSpan = 2 * W * S, NT = 32 * W;      // tokens of a chunk
  const int rank = CL > 1 ? cluster_rank() : 0;
  const int64_t unit = blockIdx.x / CL, b = unit / a.strips;
  const Channels<VEC> ch((int)(unit % a.strips), a.dim);
  const int64_t row0 = b * a.length;
  const T* gate = static_cast<const T*>(a.gate) + row0 * a.ldg + ch.first;
  const T* x = static_cast<const T*>(a.x) + row0 * a.ldx + ch.first;
  T* h = static_cast<T*>(a.h) + row0 * a.dim + ch.first;
  Quad carry = a.state ? ch.state(a.state + b * a.dim + ch.first) : quad(0.f);
  const int seg = threadIdx.x >> 4;
  Raw4<T>* const slots = reinterpret_cast<Raw4<T>*>(ring) + threadIdx.x;
  Flags ahead[D > 0 ? D : 1];
  const int64_t first = (int64_t)rank * kSpan + seg * S, stride = (int64_t)kSpan * CL;
  auto start = [&](int64_t t0, int stage) {
    #pragma unroll
    for (int i = 0; i < S; ++i) {
      Raw4<T>* const to = slots + (stage * 2 * S + i) * NT;
      if (t0 + i < a.length && ch.any()) {
        ch.copy(to, gate + (t0 + i) * a.ldg);
        ch.copy(to + S * NT, x + (t0 + i) * a.ldx);
      } else {
        infinite(to[0]);
        zero(to[S * NT]);
      }
    }
    copies_commit();
  };
  #pragma unroll
  for (int d = 0; d < D; ++d) {
    start(first + d * stride, d);
    if (FLAGS) ahead[d] = ask<S>(a.starts, a.mask, row0, first + d * stride, a.length);
  }
  if (CL > 1) cluster_barrier();      // every block has begun before one writes to another
  int round = 0, stage = 0;
  int64_t t0 = first;
  for (int64_t done = 0; done < a.length; done += stride, t0 += stride, ++round) {
    if (FLAGS && D == 0) ahead[0] = ask<S>(a.starts, a.mask, row0, t0, a.length);
    Raw4<T> rg[S], rx[S];
    if constexpr (D > 0) {
      copies_wait<D - 1>();
    } else {
      #pragma unroll
      for (int i = 0; i < S; ++i) {
        infinite(rg[i]);
        zero(rx[i]);
        if (t0 + i < a.length && ch.any()) {
          ch.load(rg[i], gate + (t0 + i) * a.ldg);
          ch.load(rx[i], x + (t0 + i) * a.ldx);
        }
      }
    }
    Quad P[S], H[S];
    Run run = {quad(1.f), quad(0.f), false};       // m: the factor, until the end
    Quad lost = quad(0.f);                          // 1 minus it
    const Flags now = FLAGS ? bits(ahead[0]) : Flags{0, 0};
    #pragma unroll
    for (int i = 0; i < S; ++i) {
      Raw4<T> gi, vi;
      if constexpr (D > 0) {
        gi = slots[(stage * 2 * S + i) * NT];
        vi = slots[(stage * 2 * S + S + i) * NT];
      } else {
        gi = rg[i];
        vi = rx[i];
      }
      if (FLAGS && !(now.live >> i & 1)) {
        infinite(gi);
        zero(vi);
      }
      const Quad g = widen(gi), xi = widen(vi);
      Quad k, u, in;
      #pragma unroll
      for (int j = 0; j < 2; ++j) {
        float2 t = mul2(g.v[j], both(-1.4426950408889634f));
        t = add2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), both(1.f));
        k.v[j] = make_float2(reciprocal_fast(t.x), reciprocal_fast(t.y));
        u.v[j] = fma2(k.v[j], both(-1.f), both(1.f));
        in.v[j] = mul2(fma2(u.v[j], both(a.mix), both(1.f - a.mix)), xi.v[j]);
      }
      if (FLAGS && (now.starts >> i & 1)) {
        run.m = run.H = quad(0.f);
        run.cut = true;
      }
      run.m = mul(run.m, k);
      run.H = fma(k, run.H, in);
      lost = fma(k, lost, u);
      P[i] = run.m;
      H[i] = run.H;
    }
    run.m = shares(run.m, lost);
    if constexpr (D > 0) {
      start(t0 + D * stride, stage);
      stage = stage + 1 == D ? 0 : stage + 1;
      if (FLAGS) {
        #pragma unroll
        for (int d = 0; d + 1 < D; ++d) ahead[d] = ahead[d + 1];
        ahead[D - 1] = ask<S>(a.starts, a.mask, row0, t0 + D * stride, a.length);
      }
    }
    Quad front = join_runs<W, CL, FLAGS, false>(sh, run, carry, round);
    #pragma unroll
    for (int i = 0; i < S; ++i) {
      if (FLAGS && (now.starts >> i & 1)) front = quad(0.f);
      if (t0 + i < a.length && ch.any()) ch.store(h + (t0 + i) * a.dim, fma(P[i], front, H[i]));
    }
  }
  if (a.last && rank == 0 && seg == 0) ch.put_state(a.last + b * a.dim + ch.first, carry);
}

template <typename T, int W, int S, int CL, int D, bool VEC>
cudaError_t scan_with(const Scan& a, int64_t strips, cudaStream_t s) {
  constexpr size_t smem = (size_t)D * 2 * S * 32 * W * sizeof(Raw4<T>);
  constexpr auto plain = scan_kernel<T, W, S, CL, D, VEC, false>, flags = scan_kernel<T, W, S, CL, D, VEC, true>;
  if (a.starts || a.mask) {
    if (const cudaError_t e = smem ? allow_shared<flags>(smem) : cudaSuccess) return e;
    return launch_strips<CL>(flags, strips, 32 * W, smem, s, a);
  }
  if (const cudaError_t e = smem ? allow_shared<plain>(smem) : cudaSuccess) return e;
  return launch_strips<CL>(plain, strips, 32 * W, smem, s, a);
}

template <typename T, bool VEC> cudaError_t scan_by_size(const Scan& a, int64_t strips, cudaStream_t s) {
  constexpr int S = sizeof(T) == 2 ? 8 : 4, D = VEC ? 3 : 0;
  if (a.length <= 2 * S) return scan_with<T, 1, S, 1, 0, VEC>(a, strips, s);
  if (a.length <= 8 * S) return scan_with<T, 4, S, 1, 0, VEC>(a, strips, s);
  if (strips >= 304 || a.length <= 16 * S) return scan_with<T, 8, S, 1, D, VEC>(a, strips, s);
  if (strips >= 76 || a.length <= 64 * S) return scan_with<T, 8, S, 4, D, VEC>(a, strips, s);
  return scan_with<T, 8, S, 8, D, VEC>(a, strips, s);
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_gated_scan(int64_t batch, int64_t length, int64_t dim, int dtype,
                                       const void* gate, int64_t ldg, const void* x, int64_t ldx,
                                       const float* state, const uint8_t* starts,
                                       const uint8_t* token_mask, int mix, void* h, float* last,
                                       void* stream) {
  const muon_status st = check_scan(batch, length, dim, dtype);
  if (st != MUON_OK) return st;
  if (ldg < 0 || ldx < 0 || (batch > 0 && length > 0 && (!gate || !x || !h))) return MUON_ERR_INVALID_ARG;
  const size_t es = size_of(dtype);
  if (any_off(es, gate, x, h) || any_off(4, state, last)) return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (batch == 0) return MUON_OK;
  NvtxRange range("muon_gated_scan");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int strips = (int)((dim + kStrip - 1) / kStrip);
  const Scan a = {length, dim, ldg, ldx, strips, mix ? 1.f : 0.f, gate, x, state, starts, token_mask, h, last};
  const int64_t rows = batch * length;
  const bool vec = dim % 4 == 0 && fours(gate, rows, ldg, es) && fours(x, rows, ldx, es) && !off(h, 4 * es);
  const cudaError_t e = by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return vec ? scan_by_size<T, true>(a, batch * strips, s) : scan_by_size<T, false>(a, batch * strips, s);
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
