// santa_visible.cuh -- which keys a decode query sees: the first `sinks` of its sequence
// and the last `window`; of a sequence behind a shared prefix, those from `first` on.
#pragma once

#include "santa_serving.h"

namespace santa {

struct Visible {
    int L;   // keys of the sequence
    int s;   // visible sinks
    int lo;  // first key of the window, >= s
};
__device__ __forceinline__ Visible visible(int L, int window, int sinks, int first) {
    Visible v;
    v.L = L;
    v.s = min(sinks, L);
    v.lo = max(max(v.s, first), L - window);
    return v;
}

}  // namespace santa
