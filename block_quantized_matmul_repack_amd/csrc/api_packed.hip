// tq_packed: calls with their arguments in an array of 64-bit slots, for bindings
// that pay for every argument of a foreign call (about 0.15 us each through
// ctypes: of 30, as much as the launch takes).
#include <utility>

#include "tq_internal.h"

namespace {

// Slot i as an argument: numbers and addresses as they are, a float in the low half.
template <typename T> T slot(const int64_t *v, size_t i)
{
    if constexpr (std::is_same_v<T, float>)
        return __builtin_bit_cast(float, (uint32_t)v[i]);
    else
        return (T)v[i];
}

template <typename... A, size_t... I>
int spread(int (*f)(A...), const int64_t *v, std::index_sequence<I...>)
{
    return f(slot<A>(v, I)...);
}

template <typename... A> int call(int (*f)(A...), const int64_t *v)
{
    return spread(f, v, std::index_sequence_for<A...>());
}

}  // namespace

extern "C" int tq_packed(int which, const int64_t *v)
{
    if (!v)
        return TQ_E_NULL;
    switch (which) {
    case TQ_CALL_TREE_ATTENTION: return call(tq_tree_attention, v);
    case TQ_CALL_TREE_ATTENTION_HEADS: return call(tq_tree_attention_heads, v);
    case TQ_CALL_PLAN_STEP: return call(tq_plan_step, v);
    case TQ_CALL_RELEASE_PAGES: return call(tq_release_pages, v);
    case TQ_CALL_RESIDUAL_NORM: return call(tq_residual_norm, v);
    case TQ_CALL_SAMPLE: return call(tq_sample, v);
    case TQ_CALL_SAMPLE_PROBS: return call(tq_sample_probs, v);
    case TQ_CALL_CACHE_BOUNDS: return call(tq_cache_bounds, v);
    case TQ_CALL_SELECT_PAGES: return call(tq_select_pages, v);
    }
    return TQ_E_TYPE;
}
