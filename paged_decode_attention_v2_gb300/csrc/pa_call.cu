// pa_call: calls with their arguments in an array of 64-bit words (a binding's
// foreign call of 34 arguments costs microseconds, one of two a tenth of that).
#include <string.h>

#include <utility>

#include "pa.h"

namespace {

template <typename A>
struct Word {
  static bool fits(const char *at) {  // (an int beyond 32 bits is refused, not cut)
    long long w;
    memcpy(&w, at, 8);
    return static_cast<long long>(static_cast<A>(w)) == w;
  }
  static A get(const char *at) {
    unsigned long long w;
    memcpy(&w, at, 8);
    return static_cast<A>(w);
  }
};
template <typename A>
struct Word<A *> {
  static bool fits(const char *) { return true; }
  static A *get(const char *at) {
    A *p;
    memcpy(&p, at, sizeof p);
    return p;
  }
};
template <>
struct Word<float> {
  static bool fits(const char *) { return true; }
  static float get(const char *at) {
    double d;
    memcpy(&d, at, 8);
    return static_cast<float>(d);
  }
};

template <typename... A, size_t... I>
pa_status_t apply(pa_status_t (*fn)(A...), const char *words, std::index_sequence<I...>) {
  if (!(Word<A>::fits(words + 8 * I) && ...)) return PA_ERR_INVALID_ARG;
  return fn(Word<A>::get(words + 8 * I)...);
}
template <typename... A>
pa_status_t apply(pa_status_t (*fn)(A...), const void *words) {
  return apply(fn, static_cast<const char *>(words), std::index_sequence_for<A...>());
}

}  // namespace

extern "C" pa_status_t pa_call(int call, const void *words) {
  if (!words) return PA_ERR_INVALID_ARG;
  switch (call) {
    case PA_CALL_Q4_APPEND: return apply(pa_q4_append, words);
    case PA_CALL_Q4_FORWARD: return apply(pa_q4_forward, words);
    case PA_CALL_LATENT_APPEND: return apply(pa_latent_append, words);
    case PA_CALL_LATENT_FORWARD: return apply(pa_latent_forward, words);
  }
  return PA_ERR_INVALID_ARG;
}
