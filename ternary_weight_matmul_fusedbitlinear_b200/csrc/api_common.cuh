// What the C ABI's source files share: error reporting, argument checks,
// workspace carving, launch timing and the quantise-then-contract sequence.
// Host only; not part of the C ABI.
#pragma once

#include "kernels.cuh"

#define MMF_CUDA(call, where)                      \
  do {                                             \
    cudaError_t e_ = (call);                       \
    if (e_ != cudaSuccess) return ::mmf::cuda_fail(e_, where); \
  } while (0)

namespace mmf {

// Set this thread's message and return `st`.
mmf_status fail(mmf_status st, const char* fmt, ...);
mmf_status cuda_fail(cudaError_t e, const char* where);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline size_t elem_bytes(mmf_dtype dt) { return dt == MMF_BF16 ? 2 : 4; }
inline bool dtype_ok(mmf_dtype dt) { return dt == MMF_F32 || dt == MMF_BF16; }
inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// Bump allocator over the caller's workspace (256-byte granules).
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <typename T> T* take(size_t count) {
    T* p = reinterpret_cast<T*>(base ? base + off : nullptr);
    off += round_up(sizeof(T) * count, 256);
    return p;
  }
};

// Per-device status word written by kernels that give up a bounded wait.
mmf_status device_status_ptr(int** out);
// The same, or null when it cannot be had.
int* status_word();

// Every launch goes through timed(): when the profiler is on, two CUDA events
// bracket it on its stream; mmf_prof_collect folds finished pairs into totals.
bool prof_is_on();
struct ProfSpan {   // holds the profiler's lock while it lives
  ProfSpan(const char* name, cudaStream_t s);
  ~ProfSpan();
  ProfSpan(const ProfSpan&) = delete;
  ProfSpan& operator=(const ProfSpan&) = delete;
  const char* name;
  cudaStream_t s;
  cudaEvent_t a, b;
};
template <class F>
cudaError_t timed(const char* name, cudaStream_t s, F&& launch) {
  if (!prof_is_on()) return launch();
  ProfSpan span(name, s);
  return launch();
}

// Quantised activations of M tokens of length K.
struct QAct {
  int8_t* q;
  float* s;
  int32_t* qsum;
};
QAct carve_qact(Carver& c, int M, int K);

mmf_status check_tlinear(const mmf_tlinear* l, const char* name);
mmf_status check_glu(const mmf_tlinear* gate, const mmf_tlinear* up, const mmf_tlinear* down, int d);
TGemmArgs gemm_args(const mmf_tlinear* const* segs, int nseg, const int8_t* q, const float* s,
                    const int32_t* qsum, int M, void* out, int ldo, const void* residual, float* h);
// The contraction `a` on the kernel that suits its size; `what` names it for the launch timing.
cudaError_t run_gemm(const TGemmArgs& a, Epi epi, mmf_dtype dt, cudaStream_t s, const char* what = "");

}  // namespace mmf
