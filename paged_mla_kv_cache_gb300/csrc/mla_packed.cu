// Calls with their arguments in an array of 8-byte words (pmg_call_packed).
#include <string.h>

#include <type_traits>
#include <utility>

#include "pmg_mla.h"

namespace {

template <class T>
T word(const void* words, size_t i) {
  const char* at = static_cast<const char*>(words) + 8 * i;
  if constexpr (std::is_floating_point<T>::value) {
    double x;
    memcpy(&x, at, 8);
    return static_cast<T>(x);
  } else {
    int64_t x;
    memcpy(&x, at, 8);
    if constexpr (std::is_pointer<T>::value) return reinterpret_cast<T>(static_cast<intptr_t>(x));
    else return static_cast<T>(x);
  }
}

template <class... A, size_t... I>
int call(int (*f)(A...), const void* words, std::index_sequence<I...>) {
  return f(word<A>(words, I)...);
}
template <class... A>
int call(int (*f)(A...), const void* words) {
  return call(f, words, std::index_sequence_for<A...>());
}

}  // namespace

extern "C" int pmg_call_packed(int which, const void* words) {
  if (words == nullptr) return PMG_ERR_NULL;
  switch (which) {
    case PMG_CALL_PLAN_STEP: return call(pmg_plan_step, words);
    case PMG_CALL_APPEND: return call(pmg_append, words);
    case PMG_CALL_LATENT_DECODE: return call(pmg_latent_decode, words);
    case PMG_CALL_LATENT_PREFILL: return call(pmg_latent_prefill, words);
    default: return PMG_ERR_ARG;
  }
}
