// The attention kernel of spec_attend_wide.cu over what the rows of a group have in common (spec_attend_shared).
#define SPEC_ATTEND_PART kCommon
#include "spec_attend_wide.cu"
