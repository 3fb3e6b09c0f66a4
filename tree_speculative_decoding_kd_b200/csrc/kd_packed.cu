// The packed form of the calls next to the verify step: one array of 8-byte values instead of
// up to 28 arguments, for bindings that pay for every argument they convert (ctypes: 5.5 us for
// 28, 1.2 with the packing; small calls behind each other gain 0.6 to 1.3 us).  Types come from
// the functions themselves.

#include <limits.h>
#include <string.h>

#include <type_traits>
#include <utility>

#include "kd_common.cuh"

namespace kd {
namespace {

// One value as a parameter of type T; *ok falls when it does not fit.
template <class T>
T take(int64_t v, bool* ok) {
  if constexpr (std::is_pointer_v<T>) {
    return reinterpret_cast<T>(static_cast<intptr_t>(v));
  } else if constexpr (std::is_same_v<T, float>) {
    double d;
    memcpy(&d, &v, sizeof d);
    return static_cast<float>(d);
  } else if constexpr (std::is_same_v<T, int>) {
    if (v < INT_MIN || v > INT_MAX) *ok = false;
    return static_cast<int>(v);
  } else {
    static_assert(std::is_same_v<T, int64_t>, "a parameter type without a packed form");
    return v;
  }
}

template <class... A, size_t... I>
int call(int (*f)(A...), const int64_t* a, std::index_sequence<I...>) {
  bool ok = true;
  ((void)take<A>(a[I], &ok), ...);
  return ok ? f(take<A>(a[I], &ok)...) : KD_EINVAL;
}

template <class... A>
int call(int (*f)(A...), const int64_t* a, int count) {
  return count == (int)sizeof...(A) ? call(f, a, std::index_sequence_for<A...>{}) : KD_EINVAL;
}

}  // namespace
}  // namespace kd

extern "C" int kd_call_packed(int op, const int64_t* args, int count) {
  if (!args) return KD_EINVAL;
  switch (op) {
    case KD_OP_QK_NORM_ROPE: return kd::call(kd_qk_norm_rope, args, count);
    case KD_OP_KV_NORM_ROPE_WRITE: return kd::call(kd_kv_norm_rope_write, args, count);
    case KD_OP_KV_NORM_ROPE_WRITE_PAGED: return kd::call(kd_kv_norm_rope_write_paged, args, count);
    case KD_OP_PROMPT_ATTN: return kd::call(kd_prompt_attn, args, count);
    case KD_OP_KV_ATTN_WEIGHTS: return kd::call(kd_kv_attn_weights, args, count);
    case KD_OP_KV_ATTN_WEIGHTS_PAGED: return kd::call(kd_kv_attn_weights_paged, args, count);
    case KD_OP_KV_EVICT: return kd::call(kd_kv_evict, args, count);
    case KD_OP_KV_EVICT_PAGED: return kd::call(kd_kv_evict_paged, args, count);
    default: return KD_EINVAL;
  }
}
