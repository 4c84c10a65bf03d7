// Gradient of the gated linear recurrence: the same joins from the last token to the
// first, over what reaches the state behind each token, c -> a (dh + c).
//
// Measured: [8, 4096, 4096] bf16 with starts 292 us, 5.5 TB/s; [4, 8192, 2048] fp32 259 us, 6.2
// TB/s; [142, 4255, 64] bf16 77 us, 6.0 TB/s; [2, 8192, 2048] bf16 93 us, 4.3 TB/s.  The larger
// ones are bound by instructions: 43 an element in 16 bits, a third of them joins.
#include "scan.cuh"

#include <algorithm>

namespace muon {

namespace {

struct ScanBwd {
  int64_t length, dim;
  uint32_t lddh, ldg, ldx, ldh;
  int strips;
  float mix;          // 1 or 0: how much of x the state's difference has
  const void *dh, *gate, *x, *h;
  const float *state, *dlast;
  const uint8_t *starts, *mask;
  void *dgate, *dx;
  float* dstate;
};

template <typename T, int W, int S, int CL, int D, int HOW, bool FLAGS>
__global__ void __launch_bounds__(32 * W, (kScanBlocks<T, W, 4, S>))
scan_bwd_kernel(const __grid_constant__ ScanBwd a) {
  extern __shared__ uint4 ring[];
  __shared__ RunSlots<W, CL> sh;
  pdl_wait();
  constexpr int kSpan = 2 * W * S;
  const int rank = CL > 1 ? cluster_rank() : 0;      // rank 0 has the last chunk
  const int64_t unit = blockIdx.x / CL, b = unit / a.strips;
  const Channels<T, HOW> ch((int)(unit % a.strips), a.dim);
  const int64_t row0 = b * a.length;
  const int seg = threadIdx.x >> 4, length = (int)a.length;
  const int chunks = (int)((a.length + kSpan - 1) / kSpan), rounds = (chunks + CL - 1) / CL;
  // the segment's first token (in front of the sequence in the last round of some ranks)
  // of the chunk to read next, and of the one to write
  int t_in = (int)((int64_t)(chunks - 1 - rank) * kSpan + seg * S), t0 = t_in;
  const int channel = D > 0 ? ch.strip : ch.first;
  const T* dh = static_cast<const T*>(a.dh) + (row0 + t_in) * (int64_t)a.lddh + channel;
  const T* gate = static_cast<const T*>(a.gate) + (row0 + t_in) * (int64_t)a.ldg + channel;
  const T* x = static_cast<const T*>(a.x) + (row0 + t_in) * (int64_t)a.ldx + channel;
  const T* h = static_cast<const T*>(a.h) + (row0 + t_in - 1) * (int64_t)a.ldh + channel;
  const int64_t out = row0 * a.dim + ch.first;
  const bool mix = a.mix != 0.f;
  if (threadIdx.x < 16)
    sh.carry[0][threadIdx.x] = four(a.dlast ? ch.state(a.dlast + b * a.dim + ch.first) : quad(0.f));
  const Ring<T, HOW, 4, S, W> slots(ring, ch.strip, a.dim);
  static_assert(kSpan % slots.kPiece == 0 || D == 0, "a row is as far ahead of its piece in every chunk");
  const T *const dh0 = dh, *const gate0 = gate, *const x0 = x, *const h0 = h;
  Flags ahead[D > 0 ? D : 1];
  auto ask_next = [&] { return ask<S>(a.starts, a.mask, row0, t_in, length); };
  auto advance = [&] {
    dh -= (uint64_t)a.lddh * (kSpan * CL);
    gate -= (uint64_t)a.ldg * (kSpan * CL);
    x -= (uint64_t)a.ldx * (kSpan * CL);
    h -= (uint64_t)a.ldh * (kSpan * CL);
    t_in -= kSpan * CL;
  };
  // how many of a segment's tokens are inside, all from its first on (chunks start at 0)
  auto inside = [&](int t) { return t < 0 ? 0 : max(0, min(S, length - t)); };
  auto start = [&](int stage) {
    const int n = inside(t_in);
    slots.arrived();
    if (n == S && t_in > 0 && mix) {
      #pragma unroll
      for (int i = 0; i < S; i += slots.kAtOnce) {
        slots.copy(stage, 0, dh, a.lddh, i, 0, S);
        slots.copy(stage, 1, gate, a.ldg, i, 0, S);
        slots.copy(stage, 2, x, a.ldx, i, 0, S);
        slots.copy(stage, 3, h, a.ldh, i, 0, S);
      }
      slots.copy_ends(stage, 0, dh, a.lddh, 0, S);
      slots.copy_ends(stage, 1, gate, a.ldg, 0, S);
      slots.copy_ends(stage, 2, x, a.ldx, 0, S);
      slots.copy_ends(stage, 3, h, a.ldh, 0, S);
    } else {
      slots.copy_some(stage, 0, dh, a.lddh, 0, n, false);
      slots.copy_some(stage, 1, gate, a.ldg, 0, n, true);
      slots.copy_some(stage, 2, x, a.ldx, 0, mix ? n : 0, false);
      slots.copy_some(stage, 3, h, a.ldh, t_in > 0 ? 0 : 1, n, false);
    }
    copies_commit();
  };
  #pragma unroll
  for (int d = 0; d < D; ++d) {
    if (d < rounds) start(d);
    else copies_commit();
    if (FLAGS) ahead[d] = ask_next();
    advance();
  }
  if (CL > 1) cluster_barrier();      // every block has begun before one writes to another
  int stage = 0;
  for (int round = 0; round < rounds; ++round) {
    Raw4<T> rd[S], rg[S], rx[S], rh[S];
    if constexpr (D > 0) {
      copies_wait<D - 1>();
      slots.arrived();
    } else {
      if (FLAGS) ahead[0] = ask_next();
      const int n = ch.any() ? inside(t_in) : 0;
      #pragma unroll
      for (int i = 0; i < S; ++i) {
        zero(rd[i]);
        infinite(rg[i]);
        zero(rx[i]);
        zero(rh[i]);
        if (i < n) {
          ch.load(rd[i], dh + (uint64_t)a.lddh * i);
          ch.load(rg[i], gate + (uint64_t)a.ldg * i);
          if (mix) ch.load(rx[i], x + (uint64_t)a.ldx * i);
          if (i > 0 || t_in > 0) ch.load(rh[i], h + (uint64_t)a.ldh * i);
        }
      }
      advance();
    }
    Quad keep[S], take[S], d[S], v[S];
    Segment run = {quad(1.f), quad(0.f), quad(0.f), false};
    const Flags now = FLAGS ? bits<S>(ahead[0]) : Flags{0, 0, true};
    auto reduce = [&](auto flagged) {
      #pragma unroll
      for (int i = S - 1; i >= 0; --i) {
        Raw4<T> di, gi, xi, hi;
        if constexpr (D > 0) {
          di = slots.get(slots.row(stage, 0, i), slots.ahead(dh0, a.lddh, i));
          gi = slots.get(slots.row(stage, 1, i), slots.ahead(gate0, a.ldg, i));
          xi = slots.get(slots.row(stage, 2, i), slots.ahead(x0, a.ldx, i));
          hi = slots.get(slots.row(stage, 3, i), slots.ahead(h0, a.ldh, i));
        } else {
          di = rd[i];
          gi = rg[i];
          xi = rx[i];
          hi = rh[i];
        }
        if constexpr (decltype(flagged)::value) {
          gi = gate_or(gi, ones(now.live, i));
          xi = masked(xi, ones(now.live, i));
        }
        shares_of(widen(gi), keep[i], take[i]);
        d[i] = widen(di);
        v[i] = widen(hi);
        if (i == 0 && t0 == 0 && a.state && ch.any()) v[0] = ch.state(a.state + b * a.dim + ch.first);
        if constexpr (decltype(flagged)::value) v[i] = masked(v[i], ~ones(now.starts, i));
        v[i] = fma(widen(xi), quad(-a.mix), v[i]);
        run.P = mul(run.P, keep[i]);
        run.Q = fma(keep[i], run.Q, take[i]);
        run.H = mul(keep[i], add(run.H, d[i]));
        if constexpr (decltype(flagged)::value) {
          const uint32_t on = ~ones(now.starts, i);
          run.P = masked(run.P, on);
          run.H = masked(run.H, on);
        }
      }
    };
    if (FLAGS && !now.quiet) reduce(std::bool_constant<FLAGS>());
    else reduce(std::false_type());
    run.cut = now.starts != 0;
    Quad c = join_segments<W, CL, FLAGS, true>(sh, run, round, [&] {
      if constexpr (D > 0) {
        if (round + D < rounds) start(stage);
        else copies_commit();      // an empty group, for the count of those in flight
        stage = stage + 1 == D ? 0 : stage + 1;
        if (FLAGS) {
          #pragma unroll
          for (int k = 0; k + 1 < D; ++k) ahead[k] = ahead[k + 1];
          ahead[D - 1] = ask_next();
        }
        advance();
      }
    });
    const int n = ch.any() ? inside(t0) : 0;
    T* const dx = static_cast<T*>(a.dx) + out + t0 * a.dim;
    T* const dg = static_cast<T*>(a.dgate) + out + t0 * a.dim;
    // what a token does with what reaches it, and what it passes on
    auto finish = [&](int i, Quad& gx, Quad& gg) {
      const Quad l = add(d[i], c), u = mul(take[i], l);
      c = mul(keep[i], l);
      gx = mix ? u : l;
      gg = mul(mul(u, keep[i]), v[i]);
    };
    Quad gx, gg;
    if (n == S && a.dx && a.dgate && (!FLAGS || now.quiet)) {
      #pragma unroll
      for (int i = S - 1; i >= 0; --i) {
        finish(i, gx, gg);
        ch.store(dx + (uint64_t)(uint32_t)a.dim * i, gx);
        ch.store(dg + (uint64_t)(uint32_t)a.dim * i, gg);
      }
    } else {
      #pragma unroll
      for (int i = S - 1; i >= 0; --i) {
        finish(i, gx, gg);
        if (FLAGS) {
          const uint32_t live = ones(now.live, i);
          gx = masked(gx, live);
          gg = masked(gg, live);
          c = masked(c, ~ones(now.starts, i));
        }
        if (i < n && a.dx) ch.store(dx + (uint64_t)(uint32_t)a.dim * i, gx);
        if (i < n && a.dgate) ch.store(dg + (uint64_t)(uint32_t)a.dim * i, gg);
      }
    }
    t0 -= kSpan * CL;
  }
  if (a.dstate && rank == 0) {
    __syncthreads();
    if (threadIdx.x < 16) ch.put_state(a.dstate + b * a.dim + ch.first, quad(sh.carry[rounds & 1][threadIdx.x]));
  }
}

constexpr int kShortThreads = 128, kShortAhead = 2;
// Short sequences, as in the forward pass
template <typename T, int HOW, bool FLAGS>
__global__ void __launch_bounds__(kShortThreads)
scan_short_bwd_kernel(const __grid_constant__ ScanBwd a, int64_t units) {
  pdl_wait();
  const int64_t unit = (int64_t)blockIdx.x * (kShortThreads / 16) + (threadIdx.x >> 4);
  if (unit >= units) return;
  const int64_t b = unit / a.strips, row0 = b * a.length;
  const Channels<T, HOW> ch((int)(unit % a.strips), a.dim);
  if (!ch.any()) return;
  const T* dh = static_cast<const T*>(a.dh) + row0 * (int64_t)a.lddh + ch.first;
  const T* gate = static_cast<const T*>(a.gate) + row0 * (int64_t)a.ldg + ch.first;
  const T* x = static_cast<const T*>(a.x) + row0 * (int64_t)a.ldx + ch.first;
  const T* h = static_cast<const T*>(a.h) + row0 * (int64_t)a.ldh + ch.first;
  T* dx = static_cast<T*>(a.dx) + row0 * a.dim + ch.first;
  T* dg = static_cast<T*>(a.dgate) + row0 * a.dim + ch.first;
  const bool mix = a.mix != 0.f;
  Quad c = a.dlast ? ch.state(a.dlast + b * a.dim + ch.first) : quad(0.f);
  for (int t0 = (int)a.length - 1; t0 >= 0; t0 -= kShortAhead) {
    Raw4<T> rd[kShortAhead], rg[kShortAhead], rx[kShortAhead], rh[kShortAhead];
    bool live[kShortAhead], begins[kShortAhead];
    #pragma unroll
    for (int i = 0; i < kShortAhead; ++i) {
      const int t = t0 - i;
      if (t < 0) continue;
      zero(rx[i]);
      zero(rh[i]);
      ch.load(rd[i], dh + t * (int64_t)a.lddh);
      ch.load(rg[i], gate + t * (int64_t)a.ldg);
      if (mix) ch.load(rx[i], x + t * (int64_t)a.ldx);
      if (t > 0) ch.load(rh[i], h + (t - 1) * (int64_t)a.ldh);
      if (FLAGS) {
        live[i] = !a.mask || a.mask[row0 + t];
        begins[i] = a.starts && a.starts[row0 + t];
      }
    }
    #pragma unroll
    for (int i = 0; i < kShortAhead; ++i) {
      const int t = t0 - i;
      if (t < 0) continue;
      Quad keep, take, v = widen(rh[i]);
      shares_of(widen(rg[i]), keep, take);
      if (t == 0 && a.state) v = ch.state(a.state + b * a.dim + ch.first);
      if (FLAGS && begins[i]) v = quad(0.f);
      v = fma(widen(rx[i]), quad(-a.mix), v);
      const Quad l = add(widen(rd[i]), c), u = mul(take, l);
      Quad gx = mix ? u : l, gg = mul(mul(u, keep), v);
      c = mul(keep, l);
      if (FLAGS && begins[i]) c = quad(0.f);
      if (FLAGS && !live[i]) {
        gx = gg = quad(0.f);
        c = l;
      }
      if (a.dx) ch.store(dx + t * a.dim, gx);
      if (a.dgate) ch.store(dg + t * a.dim, gg);
    }
  }
  if (a.dstate) ch.put_state(a.dstate + b * a.dim + ch.first, c);
}

template <typename T, int HOW> cudaError_t scan_short_bwd(const ScanBwd& a, int64_t strips, cudaStream_t s) {
  constexpr int per = kShortThreads / 16;
  return launch_k(a.starts || a.mask ? scan_short_bwd_kernel<T, HOW, true> : scan_short_bwd_kernel<T, HOW, false>,
                  dim3((unsigned)((strips + per - 1) / per)), dim3(kShortThreads), 0, s, true, a, strips);
}

template <typename T, int W, int S, int CL, int D, int HOW>
cudaError_t scan_bwd_with(const ScanBwd& a, int64_t strips, cudaStream_t s) {
  constexpr size_t smem = D * Ring<T, HOW, 4, S, W>::kStage;
  constexpr auto plain = scan_bwd_kernel<T, W, S, CL, D, HOW, false>,
                 flags = scan_bwd_kernel<T, W, S, CL, D, HOW, true>;
  if (a.starts || a.mask) {
    if (const cudaError_t e = smem ? allow_shared<flags>(smem) : cudaSuccess) return e;
    return launch_cluster(flags, strips * CL, CL, 32 * W, smem, s, a);
  }
  if (const cudaError_t e = smem ? allow_shared<plain>(smem) : cudaSuccess) return e;
  return launch_cluster(plain, strips * CL, CL, 32 * W, smem, s, a);
}

// Up to four tokens, or 32 where there are strips enough for every SM's lanes, are walked one
// after the other: one token of [256, 8192] bf16 7.1 us, 37.0 through the
// joins, 16 of [64, 4096] 10.7 and 25.4
template <typename T, int HOW> cudaError_t scan_bwd_by_size(const ScanBwd& a, int64_t strips, cudaStream_t s) {
  constexpr int S = sizeof(T) == 2 ? 4 : 2;
  if (a.length <= 4 || (a.length <= 32 && strips >= 2048)) return scan_short_bwd<T, HOW>(a, strips, s);
  return scan_layout<T, S>(a.length, strips, [&](auto w, auto m, auto cl, auto d) {
    return scan_bwd_with<T, decltype(w)::value, S * decltype(m)::value, decltype(cl)::value, decltype(d)::value, HOW>(
        a, strips, s);
  });
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
  if ((lddh | ldg | ldx | ldh) >> 32) return MUON_ERR_UNSUPPORTED_SHAPE;
  const size_t es = size_of(dtype);
  if (any_off(es, dh, gate, x, h, dgate, dx) || any_off(4, state, dlast, dstate))
    return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (batch == 0) return MUON_OK;
  NvtxRange range("muon_gated_scan_backward");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int strips = (int)((dim + kStrip - 1) / kStrip);
  const ScanBwd a = {length, dim, (uint32_t)lddh, (uint32_t)ldg, (uint32_t)ldx, (uint32_t)ldh, strips, mix ? 1.f : 0.f, dh, gate, x, h, state, dlast, starts,
                     token_mask, dgate, dx, dstate};
  const int64_t rows = batch * length, units = batch * strips;
  int how = std::max({lie(dh, rows, lddh, es), lie(gate, rows, ldg, es), lie(h, rows, ldh, es),
                            lie(dgate, rows, dim, es), lie(dx, rows, dim, es), mix ? lie(x, rows, ldx, es) : (int)kFours});
  if (rows <= 1) how = std::max(how, lie(nullptr, 2, dim, es));      // whole pieces in the row itself
  const cudaError_t e = by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return by_how<T>(how, [&](auto h) { return scan_bwd_by_size<T, decltype(h)::value>(a, units, s); });
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
