// Gated linear recurrence: the forward pass.
//
// Bound by HBM where there are strips for all SMs, by the walk over chunks where there are few.
// Measured: [16, 2048, 2048] bf16 73 us, 5.5 TB/s, [4, 8192, 2048] fp32 132 to 149 us by where its
// buffers lie, 6.1 to 5.4 TB/s; [1, 65536, 2048] bf16 207 us, 3.9 TB/s (32 strips; 64 rounds of 3.2 us),
// [1, 65536, 64] 103 us (one strip, 32 rounds); [3, 2047, 1409] fp32 with flags 32 us (69 strips; eight
// rounds); one token of 48 x 2048 1.5 us.
// Rows of an odd number of bf16 channels are stored in single elements and read in pieces from
// any address: [4, 4096, 2047] 63 us, its gradient 115, where 2046 channels, in pairs, take 51 and
// 95, and 2048 take 40 and 69.
#include "scan.cuh"

#include <algorithm>

namespace muon {

namespace {

struct Scan {
  int64_t length, dim;
  uint32_t ldg, ldx;          // 32 bits: one multiply-add makes an address
  int strips;
  float mix;          // 1: the input is multiplied by 1 - a; 0: it is not
  const void *gate, *x;
  const float* state;
  const uint8_t *starts, *mask;
  void* h;
  float* last;
};

// the input's part of a step: (1 - a) x, or x
__device__ __forceinline__ Quad input_of(const Quad& take, const Quad& x, float mix) {
  return mul(fma(take, quad(mix), quad(1.f - mix)), x);
}
// One token of a walk, the state in front of it p.  With w the smaller of a and 1 - a, the new state is
// what has the larger share, changed by w times what the other differs by (in two products,
// so that far numbers do not overflow): a state that goes from call to call loses 1 - a and
// not 1 minus the rounded a.
__device__ __forceinline__ Quad walked(const Quad& g, const Quad& x, const Quad& p, bool mix) {
  Quad q;
  #pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 v = g.v[j], in = x.v[j], from = p.v[j];
    const float2 t = make_float2(exp2_fast(fabsf(v.x) * -1.4426950408889634f), exp2_fast(fabsf(v.y) * -1.4426950408889634f));
    const float2 n = add2(t, both(1.f)), w = mul2(t, make_float2(reciprocal_fast(n.x), reciprocal_fast(n.y)));
    // w of the input and -w of the state where the state has the larger share, else the other way
    const float2 of_x = make_float2(copysignf(w.x, v.x), copysignf(w.y, v.y)), of_p = mul2(of_x, both(-1.f));
    const float2 most = make_float2(!signbit(v.x) ? from.x : mix ? in.x : 0.f, !signbit(v.y) ? from.y : mix ? in.y : 0.f);
    q.v[j] = add2(most, mix ? fma2(of_x, in, mul2(of_p, from)) : fma2(of_p, from, in));
  }
  return q;
}

// W warps a block, S tokens a segment, CL blocks a cluster, D chunks in flight (0: a
// chunk is read when it is needed)
template <typename T, int W, int S, int CL, int D, int HOW, bool FLAGS>
__global__ void __launch_bounds__(32 * W, (kScanBlocks<T, W, 2, S>))
scan_kernel(const __grid_constant__ Scan a) {
  extern __shared__ uint4 ring[];
  __shared__ RunSlots<W, CL> sh;
  pdl_wait();
  constexpr int kSpan = 2 * W * S;      // tokens of a chunk
  const int rank = CL > 1 ? cluster_rank() : 0;
  const int64_t unit = blockIdx.x / CL, b = unit / a.strips;
  const Channels<T, HOW> ch((int)(unit % a.strips), a.dim);
  const int64_t row0 = b * a.length;
  const int seg = threadIdx.x >> 4, length = (int)a.length;
  const int64_t stride = (int64_t)kSpan * CL;
  const int rounds = (int)((a.length + stride - 1) / stride);
  // the chunk to read next, at the strip's first channel or at the lane's, and the one to write
  const int channel = D > 0 ? ch.strip : ch.first;
  const T* gate = static_cast<const T*>(a.gate) + (row0 + rank * kSpan) * (int64_t)a.ldg + channel;
  const T* x = static_cast<const T*>(a.x) + (row0 + rank * kSpan) * (int64_t)a.ldx + channel;
  T* h = static_cast<T*>(a.h) + (row0 + rank * kSpan + seg * S) * a.dim + ch.first;
  int left_in = length - rank * kSpan - seg * S, left = left_in;    // tokens from the segment's first on
  gate += seg * S * (int64_t)a.ldg;
  x += seg * S * (int64_t)a.ldx;
  if (threadIdx.x < 16)
    sh.carry[0][threadIdx.x] = four(a.state ? ch.state(a.state + b * a.dim + ch.first) : quad(0.f));
  const Ring<T, HOW, 2, S, W> slots(ring, ch.strip, a.dim);
  static_assert(kSpan % slots.kPiece == 0 || D == 0, "a row is as far ahead of its piece in every chunk");
  const T *const gate0 = gate, *const x0 = x;
  Flags ahead[D > 0 ? D : 1];
  auto ask_next = [&] { return ask<S>(a.starts, a.mask, row0, a.length - left_in, length); };
  auto advance = [&] {
    gate += (uint64_t)a.ldg * (kSpan * CL);
    x += (uint64_t)a.ldx * (kSpan * CL);
    left_in -= (int)stride;
  };
  auto start = [&](int stage) {
    slots.arrived();
    if (left_in >= S) {
      #pragma unroll
      for (int i = 0; i < S; i += slots.kAtOnce) {
        slots.copy(stage, 0, gate, a.ldg, i, 0, S);
        slots.copy(stage, 1, x, a.ldx, i, 0, S);
      }
      slots.copy_ends(stage, 0, gate, a.ldg, 0, S);
      slots.copy_ends(stage, 1, x, a.ldx, 0, S);
    } else {
      slots.copy_some(stage, 0, gate, a.ldg, 0, left_in, true);
      slots.copy_some(stage, 1, x, a.ldx, 0, left_in, false);
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
    Raw4<T> rg[S], rx[S];
    if constexpr (D > 0) {
      copies_wait<D - 1>();
      slots.arrived();
    } else {
      if (FLAGS) ahead[0] = ask_next();
      const int n = ch.any() ? left_in : 0;
      #pragma unroll
      for (int i = 0; i < S; ++i) {
        infinite(rg[i]);
        zero(rx[i]);
        if (i < n) {
          ch.load(rg[i], gate + (uint64_t)a.ldg * i);
          ch.load(rx[i], x + (uint64_t)a.ldx * i);
        }
      }
      advance();
    }
    Quad P[S], H[S];
    Segment run = {quad(1.f), quad(0.f), quad(0.f), false};
    const Flags now = FLAGS ? bits<S>(ahead[0]) : Flags{0, 0, true};
    // (a loop for chunks with a flag and one without, each a single run of instructions)
    auto reduce = [&](auto flagged) {
      #pragma unroll
      for (int i = 0; i < S; ++i) {
        Raw4<T> gi, vi;
        if constexpr (D > 0) {
          gi = slots.get(slots.row(stage, 0, i), slots.ahead(gate0, a.ldg, i));
          vi = slots.get(slots.row(stage, 1, i), slots.ahead(x0, a.ldx, i));
        } else {
          gi = rg[i];
          vi = rx[i];
        }
        if constexpr (decltype(flagged)::value) {
          const uint32_t live = ones(now.live, i), on = ~ones(now.starts, i);
          gi = gate_or(gi, live);
          vi = masked(vi, live);
          run.P = masked(run.P, on);
          run.H = masked(run.H, on);
        }
        Quad keep, take;
        shares_of(widen(gi), keep, take);
        P[i] = run.P = mul(run.P, keep);
        // a constant input comes out unchanged: what it adds is the same sum as what is lost
        H[i] = run.H = fma(keep, run.H, input_of(take, widen(vi), a.mix));
        run.Q = fma(keep, run.Q, take);
      }
    };
    if (FLAGS && !now.quiet) reduce(std::bool_constant<FLAGS>());
    else reduce(std::false_type());
    run.cut = now.starts != 0;
    Quad front = join_segments<W, CL, FLAGS, false>(sh, run, round, [&] {
      if constexpr (D > 0) {
        if (round + D < rounds) start(stage);
        else copies_commit();      // an empty group, for the count of those in flight
        stage = stage + 1 == D ? 0 : stage + 1;
        if (FLAGS) {
          #pragma unroll
          for (int d = 0; d + 1 < D; ++d) ahead[d] = ahead[d + 1];
          ahead[D - 1] = ask_next();
        }
        advance();
      }
    });
    const int n = ch.any() ? left : 0;
    if (n >= S && (!FLAGS || now.quiet)) {
      #pragma unroll
      for (int i = 0; i < S; ++i) ch.store(h + (uint64_t)(uint32_t)a.dim * i, fma(P[i], front, H[i]));
    } else {
      #pragma unroll
      for (int i = 0; i < S; ++i) {
        if (FLAGS) front = masked(front, ~ones(now.starts, i));
        const Quad q = fma(P[i], front, H[i]);
        if (i < n) ch.store(h + (uint64_t)(uint32_t)a.dim * i, q);
      }
    }
    h += stride * a.dim;
    left -= (int)stride;
  }
  if (a.last && rank == 0) {
    __syncthreads();
    if (threadIdx.x < 16) ch.put_state(a.last + b * a.dim + ch.first, quad(sh.carry[rounds & 1][threadIdx.x]));
  }
}

constexpr int kShortThreads = 128, kShortAhead = 4;
// Short sequences: 16 lanes walk a strip's tokens, four of them in flight
template <typename T, int HOW, bool FLAGS>
__global__ void __launch_bounds__(kShortThreads) scan_short_kernel(const __grid_constant__ Scan a, int64_t units) {
  pdl_wait();
  const int64_t unit = (int64_t)blockIdx.x * (kShortThreads / 16) + (threadIdx.x >> 4);
  if (unit >= units) return;
  const int64_t b = unit / a.strips, row0 = b * a.length;
  const Channels<T, HOW> ch((int)(unit % a.strips), a.dim);
  if (!ch.any()) return;
  const int length = (int)a.length;
  const T* gate = static_cast<const T*>(a.gate) + row0 * (int64_t)a.ldg + ch.first;
  const T* x = static_cast<const T*>(a.x) + row0 * (int64_t)a.ldx + ch.first;
  T* h = static_cast<T*>(a.h) + row0 * a.dim + ch.first;
  Quad p = a.state ? ch.state(a.state + b * a.dim + ch.first) : quad(0.f);
  for (int t0 = 0; t0 < length; t0 += kShortAhead) {
    Raw4<T> rg[kShortAhead], rx[kShortAhead];
    bool live[kShortAhead], begins[kShortAhead];
    #pragma unroll
    for (int i = 0; i < kShortAhead; ++i) {
      const int t = t0 + i;
      if (t >= length) continue;
      ch.load(rg[i], gate + t * (int64_t)a.ldg);
      ch.load(rx[i], x + t * (int64_t)a.ldx);
      if (FLAGS) {
        live[i] = !a.mask || a.mask[row0 + t];
        begins[i] = a.starts && a.starts[row0 + t];
      }
    }
    #pragma unroll
    for (int i = 0; i < kShortAhead; ++i) {
      const int t = t0 + i;
      if (t >= length) continue;
      Quad q = p;
      if (FLAGS && begins[i]) q = quad(0.f);
      q = walked(widen(rg[i]), widen(rx[i]), q, a.mix != 0.f);
      if (!FLAGS || live[i]) p = q;
      ch.store(h + t * a.dim, p);
    }
  }
  if (a.last) ch.put_state(a.last + b * a.dim + ch.first, p);
}

template <typename T, int HOW> cudaError_t scan_short(const Scan& a, int64_t strips, cudaStream_t s) {
  constexpr int per = kShortThreads / 16;
  return launch_k(a.starts || a.mask ? scan_short_kernel<T, HOW, true> : scan_short_kernel<T, HOW, false>,
                  dim3((unsigned)((strips + per - 1) / per)), dim3(kShortThreads), 0, s, true, a, strips);
}

template <typename T, int W, int S, int CL, int D, int HOW>
cudaError_t scan_with(const Scan& a, int64_t strips, cudaStream_t s) {
  constexpr size_t smem = D * Ring<T, HOW, 2, S, W>::kStage;
  constexpr auto plain = scan_kernel<T, W, S, CL, D, HOW, false>, flags = scan_kernel<T, W, S, CL, D, HOW, true>;
  if (a.starts || a.mask) {
    if (const cudaError_t e = smem ? allow_shared<flags>(smem) : cudaSuccess) return e;
    return launch_cluster(flags, strips * CL, CL, 32 * W, smem, s, a);
  }
  if (const cudaError_t e = smem ? allow_shared<plain>(smem) : cudaSuccess) return e;
  return launch_cluster(plain, strips * CL, CL, 32 * W, smem, s, a);
}

// Up to four tokens, or 32 where there are strips enough for every SM's lanes, are walked one
// after the other: one token of [256, 8192] bf16 5.7 us, 38.0 through the joins, 16 of [64, 4096] 6.3 and 9.2
template <typename T, int HOW> cudaError_t scan_by_size(const Scan& a, int64_t strips, cudaStream_t s) {
  constexpr int S = sizeof(T) == 2 ? 8 : 4;
  if (a.length <= 4 || (a.length <= 32 && strips >= 2048)) return scan_short<T, HOW>(a, strips, s);
  return scan_layout<T, S>(a.length, strips, [&](auto w, auto m, auto cl, auto d) {
    return scan_with<T, decltype(w)::value, S * decltype(m)::value, decltype(cl)::value, decltype(d)::value, HOW>(
        a, strips, s);
  });
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
  if ((ldg | ldx) >> 32) return MUON_ERR_UNSUPPORTED_SHAPE;
  const size_t es = size_of(dtype);
  if (any_off(es, gate, x, h) || any_off(4, state, last)) return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (batch == 0) return MUON_OK;
  NvtxRange range("muon_gated_scan");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int strips = (int)((dim + kStrip - 1) / kStrip);
  const Scan a = {length, dim, (uint32_t)ldg, (uint32_t)ldx, strips, mix ? 1.f : 0.f, gate, x, state, starts, token_mask, h, last};
  const int64_t rows = batch * length, units = batch * strips;
  int how = std::max({lie(gate, rows, ldg, es), lie(x, rows, ldx, es), lie(h, rows, dim, es)});
  if (rows <= 1) how = std::max(how, lie(nullptr, 2, dim, es));      // whole pieces in the row itself
  const cudaError_t e = by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return by_how<T>(how, [&](auto h) { return scan_by_size<T, decltype(h)::value>(a, units, s); });
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
