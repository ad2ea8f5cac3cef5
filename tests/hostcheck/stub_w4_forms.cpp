// The stand-ins of stub_w4_launchers.cpp, and which forms the library holds.
// Test infrastructure: never part of libqlin.so.
#include "stub_w4_launchers.cpp"

extern "C" int w4_forms(void) { return qlin::kW4Forms; }
extern "C" int w4_first_tiled(void) { return qlin::kW4Tiled64x8; }
extern "C" int w4_form_built(int form, int group, int pair) { return qlin::w4_form_built(form, group, pair != 0); }
