// Linear attention with one decay per head, over ragged histories.
//
//   S_t = decay S_(t-1) + k_t v_t^T,   o_t = scale q_t S_t
//
// and its gradient, which is the same map three times.  With U_t the gradient
// of S_t, U_t = scale q_t do_t^T + W_t and W_(t-1) = decay U_t:
//   dq_t = scale S_t do_t  : attention of (do, v, k), forwards, state S^T
//   dk_t = U_t v_t         : attention of (v, do, q), backwards, state U^T
//   dv_t = U_t^T k_t       : attention of (k, q, do), backwards, state U
// A role says which tensors stand where; `lead` is 1 where the state decays
// before a step's product is added (S) and 0 where it does after it (W).
#include "common.hpp"
#include "rows.hpp"

namespace dlrm {
namespace {

struct Strided {
  const void* p;
  int64_t ts, hs;  // row and head strides, in elements
};
struct Role {
  Strided q, k, v, o;      // o is written
  const float* first;      // nullable: the state before the first step
  float* last;             // nullable: the state after the last step
  int dk, dv;              // this role's contraction and output widths
  int flip;                // states in memory are transposed: [dv][dk]
  int back;                // time runs from a history's end to its start
  float kscale, oscale;    // on every k, and on the output
};
struct Roles {
  Role r[3];
};

// One block per history, head and role: the recurrence as it stands.
template <class T>
__global__ __launch_bounds__(128) void linattn_kernel(Roles roles, const int64_t* __restrict__ offsets, int H,
                                                      const float* __restrict__ decay) {
  __shared__ float S[128 * 128];
  __shared__ float qs[128], ks[128];
  const Role r = roles.r[blockIdx.y];
  const int64_t b = blockIdx.x / H;
  const int h = blockIdx.x - (int)b * H, j = threadIdx.x;
  const int64_t beg = offsets[b], len = offsets[b + 1] - beg;
  const float lam = decay[h];
  const int64_t sb = (b * H + h) * r.dk * r.dv;
  auto at = [&](int i) { return r.flip ? j * r.dk + i : i * r.dv + j; };
  if (j < r.dv)
    for (int i = 0; i < r.dk; ++i) S[i * 128 + j] = r.first ? r.first[sb + at(i)] : 0.f;
  for (int64_t s = 0; s < len; ++s) {
    const int64_t t = beg + (r.back ? len - 1 - s : s);
    __syncthreads();
    if (j < r.dk) {
      qs[j] = to_f32(static_cast<const T*>(r.q.p)[t * r.q.ts + h * r.q.hs + j]);
      ks[j] = to_f32(static_cast<const T*>(r.k.p)[t * r.k.ts + h * r.k.hs + j]) * r.kscale;
    }
    __syncthreads();
    if (j >= r.dv) continue;
    const float v = to_f32(static_cast<const T*>(r.v.p)[t * r.v.ts + h * r.v.hs + j]);
    float acc = 0.f;
    for (int i = 0; i < r.dk; ++i) {
      const float u = (r.back ? 1.f : lam) * S[i * 128 + j] + ks[i] * v;
      acc += qs[i] * u;
      S[i * 128 + j] = r.back ? lam * u : u;
    }
    static_cast<T*>(const_cast<void*>(r.o.p))[t * r.o.ts + h * r.o.hs + j] = from_f32<T>(acc * r.oscale);
  }
  if (r.last && j < r.dv)
    for (int i = 0; i < r.dk; ++i) r.last[sb + at(i)] = S[i * 128 + j];
}

template <class T>
__global__ __launch_bounds__(128) void linattn_step_kernel(Strided q, Strided k, Strided v, Strided o, int H, int dk,
                                                           int dv, const float* __restrict__ decay, float scale,
                                                           float* __restrict__ state,
                                                           const int64_t* __restrict__ slots) {
  const int64_t b = blockIdx.x / H;
  const int h = blockIdx.x - (int)b * H, j = threadIdx.x;
  if (j >= dv) return;
  const int64_t slot = slots ? slots[b] : b;
  float acc = 0.f;
  if (slot >= 0) {
    float* S = state + (slot * H + h) * dk * dv;
    const T* qp = static_cast<const T*>(q.p) + b * q.ts + h * q.hs;
    const T* kp = static_cast<const T*>(k.p) + b * k.ts + h * k.hs;
    const float vj = to_f32(static_cast<const T*>(v.p)[b * v.ts + h * v.hs + j]), lam = decay[h];
    for (int i = 0; i < dk; ++i) {
      const float u = lam * S[i * dv + j] + to_f32(kp[i]) * vj;
      S[i * dv + j] = u;
      acc += to_f32(qp[i]) * u;
    }
  }
  static_cast<T*>(const_cast<void*>(o.p))[b * o.ts + h * o.hs + j] = from_f32<T>(acc * scale);
}

bool head_ok(int32_t w) { return w >= 8 && w <= 128 && w % 8 == 0; }
bool strided_ok(const Strided& s) { return s.p && aligned16(s.p) && s.ts % 8 == 0 && s.hs % 8 == 0; }
bool state_ok(const float* p) { return aligned16(p); }

// shared by the forward and backward calls
int check_shape(int32_t dtype, const int64_t* offsets, int64_t B, int32_t H, int64_t max_len, int32_t dk, int32_t dv,
                const float* decay) {
  if (!is_activation(dtype) || B < 1 || H < 1 || max_len < 0 || !head_ok(dk) || !head_ok(dv)) return DLRM_E_INVALID;
  if (!offsets || !decay) return DLRM_E_INVALID;
  if (B > 0x7fffffffLL / 32 / H) return DLRM_E_UNSUPPORTED;
  return DLRM_OK;
}

int launch(const Roles& roles, int count, int32_t dtype, const int64_t* offsets, int64_t B, int32_t H,
           const float* decay, hipStream_t stream) {
  const dim3 grid((unsigned)(B * H), (unsigned)count);
  if (dtype == DLRM_F32)
    hipLaunchKernelGGL((linattn_kernel<float>), grid, dim3(128), 0, stream, roles, offsets, H, decay);
  else
    hipLaunchKernelGGL((linattn_kernel<uint16_t>), grid, dim3(128), 0, stream, roles, offsets, H, decay);
  return launch_status();
}

}  // namespace
}  // namespace dlrm

using namespace dlrm;

extern "C" size_t dlrm_linattn_workspace_size(int64_t B, int32_t H, int64_t max_len, int32_t dk, int32_t dv) {
  (void)B; (void)H; (void)max_len; (void)dk; (void)dv;
  return 0;
}

extern "C" int dlrm_linattn_fwd(const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts, int64_t k_hs,
                                const void* v, int64_t v_ts, int64_t v_hs, int32_t dtype, const int64_t* offsets,
                                int64_t B, int32_t H, int64_t max_len, int32_t dk, int32_t dv, const float* decay,
                                float scale, const float* state0, void* o, int64_t o_ts, int64_t o_hs, float* state,
                                void* ws, size_t ws_bytes, hipStream_t stream) {
  (void)ws_bytes;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return DLRM_E_INVALID;
  const int rc = check_shape(dtype, offsets, B, H, max_len, dk, dv, decay);
  if (rc != DLRM_OK) return rc;
  const Role r{{q, q_ts, q_hs}, {k, k_ts, k_hs}, {v, v_ts, v_hs}, {o, o_ts, o_hs}, state0, state, dk, dv,
               0, 0, 1.f, scale};
  if (max_len > 0 && (!strided_ok(r.q) || !strided_ok(r.k) || !strided_ok(r.v) || !strided_ok(r.o)))
    return DLRM_E_INVALID;
  if (!state_ok(state0) || !state_ok(state)) return DLRM_E_INVALID;
  Roles roles{};
  roles.r[0] = r;
  return launch(roles, 1, dtype, offsets, B, H, decay, stream);
}

extern "C" size_t dlrm_linattn_bwd_workspace_size(int64_t B, int32_t H, int64_t max_len, int32_t dk, int32_t dv) {
  (void)B; (void)H; (void)max_len; (void)dk; (void)dv;
  return 0;
}

extern "C" int dlrm_linattn_bwd(const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts, int64_t k_hs,
                                const void* v, int64_t v_ts, int64_t v_hs, const void* do_, int64_t do_ts,
                                int64_t do_hs, int32_t dtype, const int64_t* offsets, int64_t B, int32_t H,
                                int64_t max_len, int32_t dk, int32_t dv, const float* decay, float scale,
                                const float* state0, const float* dstate, void* dq, int64_t dq_ts, int64_t dq_hs,
                                void* dk_, int64_t dk_ts, int64_t dk_hs, void* dv_, int64_t dv_ts, int64_t dv_hs,
                                float* dstate0, void* ws, size_t ws_bytes, hipStream_t stream) {
  (void)ws_bytes;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return DLRM_E_INVALID;
  const int rc = check_shape(dtype, offsets, B, H, max_len, dk, dv, decay);
  if (rc != DLRM_OK) return rc;
  const Strided Q{q, q_ts, q_hs}, K{k, k_ts, k_hs}, V{v, v_ts, v_hs}, O{do_, do_ts, do_hs};
  const Strided DQ{dq, dq_ts, dq_hs}, DK{dk_, dk_ts, dk_hs}, DV{dv_, dv_ts, dv_hs};
  if (max_len > 0)
    for (const Strided* s : {&Q, &K, &V, &O, &DQ, &DK, &DV})
      if (!strided_ok(*s)) return DLRM_E_INVALID;
  if (!state_ok(state0) || !state_ok(dstate) || !state_ok(dstate0) || (dstate0 && dstate0 == dstate))
    return DLRM_E_INVALID;
  Roles roles{};
  roles.r[0] = Role{O, V, K, DQ, state0, nullptr, dv, dk, 1, 0, 1.f, scale};
  roles.r[1] = Role{V, O, Q, DK, dstate, nullptr, dv, dk, 1, 1, scale, 1.f};
  roles.r[2] = Role{K, Q, O, DV, dstate, dstate0, dk, dv, 0, 1, scale, 1.f};
  return launch(roles, 3, dtype, offsets, B, H, decay, stream);
}

extern "C" int dlrm_linattn_step(const void* q, int64_t q_bs, int64_t q_hs, const void* k, int64_t k_bs, int64_t k_hs,
                                 const void* v, int64_t v_bs, int64_t v_hs, int32_t dtype, int64_t B, int32_t H,
                                 int32_t dk, int32_t dv, const float* decay, float scale, float* state,
                                 const int64_t* slots, void* o, int64_t o_bs, int64_t o_hs, hipStream_t stream) {
  if (!is_activation(dtype) || B < 0 || H < 1 || !head_ok(dk) || !head_ok(dv)) return DLRM_E_INVALID;
  if (B == 0) return DLRM_OK;
  const Strided Q{q, q_bs, q_hs}, K{k, k_bs, k_hs}, V{v, v_bs, v_hs}, O{o, o_bs, o_hs};
  if (!strided_ok(Q) || !strided_ok(K) || !strided_ok(V) || !strided_ok(O) || !decay || !state || !state_ok(state))
    return DLRM_E_INVALID;
  if (B > 0x7fffffffLL / 32 / H) return DLRM_E_UNSUPPORTED;
  const dim3 grid((unsigned)(B * H));
  if (dtype == DLRM_F32)
    hipLaunchKernelGGL((linattn_step_kernel<float>), grid, dim3(128), 0, stream, Q, K, V, O, H, dk, dv, decay, scale,
                       state, slots);
  else
    hipLaunchKernelGGL((linattn_step_kernel<uint16_t>), grid, dim3(128), 0, stream, Q, K, V, O, H, dk, dv, decay,
                       scale, state, slots);
  return launch_status();
}
