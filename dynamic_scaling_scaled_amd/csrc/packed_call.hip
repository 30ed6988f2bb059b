// packed_call.hip -- fp8_call_packed: the decoder-layer calls with their arguments
// as 64-bit words.  Host code only.  The parameter types are taken from the
// declarations themselves, so a call's words cannot drift from its signature.
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "fp8rt.h"

namespace {

// Reads words one after the other; `ok` falls when one does not fit its parameter.
struct Words {
  const int64_t* w;
  bool ok;

  template <typename T>
  T next() {
    if constexpr (std::is_pointer<T>::value) {
      return reinterpret_cast<T>(static_cast<intptr_t>(*w++));
    } else if constexpr (std::is_same<T, float>::value) {
      double d;
      memcpy(&d, w++, sizeof(d));
      return static_cast<float>(d);
    } else if constexpr (std::is_same<T, fp8rt_gran>::value) {
      const int32_t rows = next<int32_t>();
      return fp8rt_gran{rows, next<int32_t>()};
    } else if constexpr (sizeof(T) == 8) {
      return static_cast<T>(*w++);
    } else {  // int32_t, uint32_t and the enumerations
      const int64_t x = *w++;
      ok = ok && x >= INT32_MIN && x <= INT32_MAX;
      return static_cast<T>(static_cast<int32_t>(x));
    }
  }
};

template <typename T>
constexpr int64_t words_of() {
  return std::is_same<T, fp8rt_gran>::value ? 2 : 1;
}

template <typename... A>
fp8rt_status call(fp8rt_status (*f)(A...), const int64_t* words, int64_t n) {
  if (n != 1 + (words_of<A>() + ...)) return FP8RT_EINVAL;
  Words r{words + 1, true};
  std::tuple<A...> args{r.template next<A>()...};  // braces: left to right
  return r.ok ? std::apply(f, args) : FP8RT_EINVAL;
}

}  // namespace

extern "C" fp8rt_status fp8_call_packed(const int64_t* words, int64_t n) {
  if (!words || n < 1) return FP8RT_EINVAL;
  switch (words[0]) {
    case FP8RT_CALL_RMSNORM_QUANTIZE: return call(fp8_rmsnorm_quantize, words, n);
    case FP8RT_CALL_RMSNORM_BACKWARD: return call(fp8_rmsnorm_backward, words, n);
    case FP8RT_CALL_KV_APPEND: return call(fp8_kv_append, words, n);
    case FP8RT_CALL_PAGED_ATTENTION: return call(fp8_paged_attention, words, n);
    case FP8RT_CALL_EXPERT_ROUTE: return call(fp8_expert_route, words, n);
    case FP8RT_CALL_EXPERT_ROUTE_BACKWARD: return call(fp8_expert_route_backward, words, n);
    case FP8RT_CALL_EXPERT_GEMM: return call(fp8_expert_gemm, words, n);
    case FP8RT_CALL_GATED_QUANTIZE: return call(fp8_gated_quantize, words, n);
    case FP8RT_CALL_GATED_BACKWARD: return call(fp8_gated_backward, words, n);
    case FP8RT_CALL_EXPERT_COMBINE: return call(fp8_expert_combine, words, n);
    case FP8RT_CALL_EXPERT_COMBINE_BACKWARD: return call(fp8_expert_combine_backward, words, n);
  }
  return FP8RT_EINVAL;
}
