// Gated linear recurrence and its gradient.
#include "sequence.cuh"

namespace muon {

namespace {

constexpr int kScanThreads = 128;

struct Scan {
  int64_t length, dim, ldg, ldx;
  const void *gate, *x;
  const float* state;
  const uint8_t *starts, *mask;
  void* h;
  float* last;
};

// a = sigmoid(g) and 1 - a, each to fp32's precision: the smaller of the two is
// computed, the larger is 1 minus it.
struct Gate { float small; bool keeps; };     // keeps: a >= 1/2, small = 1 - a; else small = a
__device__ __forceinline__ Gate gate_of(float g) {
  const float t = __expf(-fabsf(g));
  return {t / (1.f + t), g >= 0.f};
}
// The state behind a token.  Written with the smaller share, the rounding of the larger
// does not change what a long run of equal gates converges to.
template <bool MIX> __device__ __forceinline__ float step(Gate a, float p, float x) {
  if (MIX) return a.keeps ? fmaf(a.small, x - p, p) : fmaf(a.small, p - x, x);
  return a.keeps ? fmaf(-a.small, p, p) + x : fmaf(a.small, p, x);
}

template <typename T, bool MIX>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const __grid_constant__ Scan a) {
  pdl_wait();
  const int64_t strips = (a.dim + kScanThreads - 1) / kScanThreads;
  const int64_t c = blockIdx.x % strips * kScanThreads + threadIdx.x, b = blockIdx.x / strips;
  if (c >= a.dim) return;
  const T* gate = static_cast<const T*>(a.gate) + b * a.length * a.ldg + c;
  const T* x = static_cast<const T*>(a.x) + b * a.length * a.ldx + c;
  T* h = static_cast<T*>(a.h) + b * a.length * a.dim + c;
  float p = a.state ? a.state[b * a.dim + c] : 0.f;
  for (int64_t t = 0; t < a.length; ++t) {
    if (!a.mask || a.mask[b * a.length + t]) {
      if (a.starts && a.starts[b * a.length + t]) p = 0.f;
      p = step<MIX>(gate_of(to_f(gate[t * a.ldg])), p, to_f(x[t * a.ldx]));
    }
    h[t * a.dim] = from_f<T>(p);
  }
  if (a.last) a.last[b * a.dim + c] = p;
}

struct ScanBwd {
  int64_t length, dim, lddh, ldg, ldx, ldh;
  const void *dh, *gate, *x, *h;
  const float *state, *dlast;
  const uint8_t *starts, *mask;
  void *dgate, *dx;
  float* dstate;
};

template <typename T, bool MIX>
__global__ void __launch_bounds__(kScanThreads) scan_bwd_kernel(const __grid_constant__ ScanBwd a) {
  pdl_wait();
  const int64_t strips = (a.dim + kScanThreads - 1) / kScanThreads;
  const int64_t c = blockIdx.x % strips * kScanThreads + threadIdx.x, b = blockIdx.x / strips;
  if (c >= a.dim) return;
  const int64_t row0 = b * a.length;
  float l = a.dlast ? a.dlast[b * a.dim + c] : 0.f;
  for (int64_t t = a.length - 1; t >= 0; --t) {
    const int64_t r = row0 + t;
    l += to_f(static_cast<const T*>(a.dh)[r * a.lddh + c]);
    float dx = 0.f, dg = 0.f;
    if (!a.mask || a.mask[r]) {
      const bool start = a.starts && a.starts[r];
      const float before = t ? to_f(static_cast<const T*>(a.h)[(r - 1) * a.ldh + c])
                             : a.state ? a.state[b * a.dim + c] : 0.f;
      const float p = start ? 0.f : before;
      const Gate g = gate_of(to_f(static_cast<const T*>(a.gate)[r * a.ldg + c]));
      const float slope = fmaf(-g.small, g.small, g.small);
      const float kept = g.keeps ? fmaf(-g.small, l, l) : g.small * l;
      const float rest = g.keeps ? g.small * l : fmaf(-g.small, l, l);
      dx = MIX ? rest : l;
      dg = slope * l * (MIX ? p - to_f(static_cast<const T*>(a.x)[r * a.ldx + c]) : p);
      l = start ? 0.f : kept;
    }
    if (a.dx) static_cast<T*>(a.dx)[r * a.dim + c] = from_f<T>(dx);
    if (a.dgate) static_cast<T*>(a.dgate)[r * a.dim + c] = from_f<T>(dg);
  }
  if (a.dstate) a.dstate[b * a.dim + c] = l;
}

muon_status check_scan(int64_t batch, int64_t length, int64_t dim, int dtype) {
  if (batch < 0 || length < 0) return MUON_ERR_INVALID_ARG;
  if (dim < 1 || dim > 1 << 20 || batch >= (int64_t)1 << 31 || length >= (int64_t)1 << 31 ||
      batch * dim >= (int64_t)1 << 33 || batch * ((dim + kScanThreads - 1) / kScanThreads) >= (int64_t)1 << 31)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  return known(dtype) ? MUON_OK : MUON_ERR_DTYPE;
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
  if (any_off(size_of(dtype), gate, x, h) || any_off(4, state, last)) return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (batch == 0) return MUON_OK;
  NvtxRange range("muon_gated_scan");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Scan a = {length, dim, ldg, ldx, gate, x, state, starts, token_mask, h, last};
  const cudaError_t e = by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return launch_k(mix ? scan_kernel<T, true> : scan_kernel<T, false>,
                    dim3((unsigned)(batch * ((dim + kScanThreads - 1) / kScanThreads))),
                    dim3(kScanThreads), 0, s, true, a);
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

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
  if (any_off(size_of(dtype), dh, gate, x, h, dgate, dx) || any_off(4, state, dlast, dstate))
    return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (batch == 0) return MUON_OK;
  NvtxRange range("muon_gated_scan_backward");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const ScanBwd a = {length, dim, lddh, ldg, ldx, ldh, dh, gate, x, h, state, dlast, starts, token_mask,
                     dgate, dx, dstate};
  const cudaError_t e = by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return launch_k(mix ? scan_bwd_kernel<T, true> : scan_bwd_kernel<T, false>,
                    dim3((unsigned)(batch * ((dim + kScanThreads - 1) / kScanThreads))),
                    dim3(kScanThreads), 0, s, true, a);
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
